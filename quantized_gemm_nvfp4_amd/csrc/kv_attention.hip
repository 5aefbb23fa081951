// Attention over the NVFP4 cache (layout: kv_cache.hip).
//
// A segment is a set of rows against a run of keys: rows are the query heads
// that share one key/value head -- (query token, head in group) pairs of one
// sequence, or of the whole batch against the shared prefix.  Rows whose keys
// are cut into several segments leave partial results (m, l, O) in the
// workspace and a second kernel joins them:
//   M = max m,  o = sum 2^(m - M) O / sum 2^(m - M) l.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "common.h"
#include "kv_cache.h"
#include "launch.h"

namespace nvfp4k {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Softmax weights are 2^(s - m + kBias), where m may lag behind the running
// maximum by kLag (fewer rescalings of the sums): at most 2^(kBias + kLag) <
// 65504, and in fp16 they keep 11 bits down to 2^-(14 + kBias) of the largest
// and are lost below 2^-(25 + kBias).
constexpr float kBias = 7.0f, kLag = 8.0f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float finite_or_zero(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// From a row's products to its scores in units of log 2, where q was scaled by
// 2^sh = 1 / (i1 i2) and e is the biased exponent of its largest magnitude (255:
// an infinity or NaN among its values).  Not below the smallest normal number:
// the product may round to zero for tiny rows or scales, and a masked score is
// -inf, whose product with zero is NaN.  Products stay below 2^35, so scores that
// the bound raises stay below 2^-91, which no weight shows.
__device__ __forceinline__ float score_factor(int e, float scale, float k_gscale, float i1, float i2) {
  const float f = (scale * i1) * (k_gscale * i2) * kLog2e;
  return e == 255 ? __builtin_nanf("") : f < 0x1p-126f ? 0x1p-126f : f;
}

// Sequence of query token t: the last b with starts[b] <= t.
__device__ __forceinline__ int sequence_of(const KvAttention& a, int t) {
  if (!a.q_starts) return t;
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.q_starts[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ int own_length(const KvAttention& a, int b) {
  return max(0, min(a.kv_lens[b], a.max_kv_len));
}

// A segment.
struct Item {
  const int32_t* pages;
  int kvh;
  int key0, key1;      // its keys, positions in the sequence or the prefix
  int q0, n, rows;     // queries of the sequence from q0 on; row x is token q0 + x / group, head kvh * group + x % group
  int row0;            // first row of this tile
  int seq;             // the sequence, or -1: the prefix (rows of every sequence)
};

// Keys of the prefix that query token t sees.
__device__ __forceinline__ int prefix_limit(const KvAttention& a, int t) {
  const int b = sequence_of(a, t);
  const int q0 = a.q_starts ? a.q_starts[b] : b, n = a.q_starts ? a.q_starts[b + 1] - q0 : 1;
  const int64_t seen = (int64_t)own_length(a, b) - n + (t - q0) + 1;       // of the sequence's own keys
  return (int)max((int64_t)0, min((int64_t)a.prefix_len, a.prefix_len + seen));
}
// Keys of its own sequence (len of them, n queries from q0 on) that query token t sees.
__device__ __forceinline__ int own_limit(int len, int q0, int n, int t) {
  return (int)max((int64_t)0, min((int64_t)len, (int64_t)len - n + (t - q0) + 1));
}

// A streaming workgroup's pass: 64 keys for each of its 4 waves.
constexpr int kPass = 256;

// How a call is cut up (host-made).
//
// The prefix is cut into prefix_chunks chunks for each row tile.  The
// sequences' own keys are one segment a sequence and row tile while that
// spreads well (workers == 0); else all passes of all sequences, row tiles and heads
// are laid end to end and dealt to workers, one on each place of the card, in
// equal consecutive shares, whatever the lengths.  A worker's share may cross
// sequences; only the segments at its two ends can be partial, so it has two
// slots for partial results: 0 for a segment begun by an earlier worker, 1
// for one that a later worker goes on with.
struct Cut {
  int prefix_chunks, prefix_chunk, prefix_tiles;
  uint32_t prefix_items;                           // workgroups of this launch that take the prefix (first)
  int own_tiles, own_rows;                         // row tiles of a sequence, rows of a tile
  int workers;
  int own_chunks, own_chunk;                       // tile kernel: chunks of a sequence's keys, keys of one
  // partial results by index: (m, l) pairs and O.  First the prefix's, [row]
  // [chunk]; then, with a prefix or several chunks, the sequences' own, [row]
  // [own_chunks] (1 for complete segments); then the workers' slots, [worker]
  // [2][own_rows].
  float* part_ml;
  float* part_o;
  int64_t full_at, slot_at;
};

// Passes of a sequence (an empty one has its zeros to write).
__device__ __forceinline__ int passes_of(int len) { return max(1, (len + kPass - 1) / kPass); }

// Inclusive sum over the wave's lanes, by data-parallel-primitive moves.
template <int kCtrl, int kRowMask>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, kCtrl, kRowMask, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v = dpp_add<0x111, 0xF>(v);      // row_shr:1, 2, 4, 8: within rows of 16
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);      // row_bcast:15 into rows 1 and 3
  return dpp_add<0x143, 0xC>(v);   // row_bcast:31 into rows 2 and 3
}

// Passes of a worker's share.
__device__ __forceinline__ int share_of(const Cut& cut, int total) { return (total + cut.workers - 1) / cut.workers; }

// A sequence's passes in the row of all passes of one head and row tile.
struct Spot {
  int all;             // passes of all sequences
  int seq, before;     // the sequence, the passes before its first
  int len;
};
// With find: of the sequence at pass position pick(all); else of sequence b.
template <bool kFind, typename Pick>
__device__ __forceinline__ Spot spot_of(const KvAttention& a, int b, Pick pick) {
  const int lane = threadIdx.x & 63;
  Spot s{0, b, 0, 0};
  auto len_at = [&](int i) { return i < a.batch ? own_length(a, i) : -1; };
  auto sum_to_here = [&](int len) { return wave_scan(len < 0 ? 0 : passes_of(len)); };
  auto take = [&](int base, int b0, int len, int end, int i) {
    s.seq = b0 + i;
    s.before = base + __builtin_amdgcn_readlane(end, i) - passes_of(__builtin_amdgcn_readlane(len, i));
    s.len = __builtin_amdgcn_readlane(len, i);
  };
  const int len0 = len_at(lane), end0 = sum_to_here(len0);
  s.all = __builtin_amdgcn_readlane(end0, 63);
  for (int b0 = 64; b0 < a.batch; b0 += 64) s.all += __builtin_amdgcn_readlane(sum_to_here(len_at(b0 + lane)), 63);
  const int x = kFind ? pick(s.all) : 0;
  int base = 0, len = len0, end = end0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    if (b0 > 0) {
      base += __builtin_amdgcn_readlane(end, 63);
      len = len_at(b0 + lane);
      end = sum_to_here(len);
    }
    if (kFind) {
      const uint64_t past = __ballot(base + end > x);
      if (past != 0) {
        take(base, b0, len, end, __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)past) - 1));
        break;
      }
    } else if (b < b0 + 64) {
      take(base, b0, len, end, b - b0);
      break;
    }
  }
  return s;
}

__device__ __forceinline__ void own_rows_of(const KvAttention& a, int group, Item& it) {
  it.pages = a.page_table + it.seq * a.table_width;
  it.q0 = a.q_starts ? max(0, a.q_starts[it.seq]) : it.seq;
  const int q1 = a.q_starts ? min((int)a.total_q, a.q_starts[it.seq + 1]) : it.seq + 1;
  it.n = max(0, q1 - it.q0);
  it.rows = min(it.n, a.max_q_len) * group;
}

// ---- few rows: keys streamed through registers ------------------------------
//
// One wave takes 64 keys at a time and up to 16 kTiles rows.  With lane =
// 16 g + r (the layout of v_mfma_f32_16x16x32_f16: operands hold row or
// column r at k = 8 g .. 8 g + 7, results column r at rows 4 g .. 4 g + 3):
//   S^T = K Q^T   tile i (of 4): row r is key 16 (r / 4) + 4 i + r % 4, so
//                 lane (g, r) ends up with query r's scores of the 16
//                 consecutive keys of fragment g -- V's fragments;
//                 contraction step s covers values D/4 g + 8 s .. + 7, so a
//                 lane's K codes are D/8 consecutive bytes;
//   O^T = V^T P^T V's fragment gives a lane the codes of one value pair for
//                 its 16 keys in 16 bytes, and P is in the lane's registers
//                 in just that order: no shuffle, no LDS.
// The conversion yields value pairs (2 p, 2 p + 1) of one key.  With one row
// tile they are contracted as they come, against (P, 0) for the even values
// and (0, P) for the odd: twice the MFMAs, which are idle here, instead of a
// permute per pair.  With more row tiles the pairs are permuted once into
// key order and serve every tile.  The sum of the weights is one more MFMA,
// against ones.
//
// The block scales of 64 keys are D/16 bytes a lane; they pass through LDS
// (the wave's own part, no barrier) because every lane needs those of other
// lanes' keys: loading them where they are used costs 8 times the requests.
//
// Loads run ahead of their use: K codes and V codes by one pass, scales by
// two (through LDS by one), page numbers by three.
//
// Bound by HBM with one row tile.  64 query on 8 key heads of 128 over 48
// sequences of 0 to 16000 keys, 488 MB: 102 us, 4.8 TB/s (a plain read reaches
// 6.2); over one of 500009, 576 MB: 112 us, 5.1 TB/s.  What is lost is the
// start, where lengths, pages and keys are loaded one after the other (2 to 3
// us, 7 to 9 while all workgroups do it), and the uneven end.
template <int D, int kTiles>
struct Stream {
  static constexpr int kWaves = 4;
  static constexpr int kRows = 16 * kTiles;
  static constexpr int kKWords = D / 32;      // dwords of K codes a lane holds per key
  static constexpr int kPairs = D / 32;       // 16-byte V loads a lane holds per fragment
  static constexpr int kSWords = D / 64;      // dwords of scales a lane loads per pass, K and V each
  // workgroups per compute unit the registers allow
  static constexpr int kOccupancy = D == 256 ? 1 : D == 64 || kTiles == 1 ? 3 : 2;
};

template <int kWords>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (kWords == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (kWords == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  }
}
template <int kWords>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t* w) {
  if constexpr (kWords == 1) *reinterpret_cast<uint32_t*>(p) = w[0];
  else if constexpr (kWords == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Two E4M3 bytes of a dword (the low or, kTwo and hi, the high pair) as fp16.
template <bool kTwo>
__device__ __forceinline__ half2v e4m3_pair(uint32_t w, int hi) {
  return kTwo && hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
                    : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
}

template <int D>
__device__ __forceinline__ uint32_t load_k_scales(const uint8_t* p) {   // D/64 bytes
  if constexpr (D == 64) return *p;
  else if constexpr (D == 128) return *reinterpret_cast<const uint16_t*>(p);
  else return *reinterpret_cast<const uint32_t*>(p);
}

// The value pairs (2 p, 2 p + 1) of 4 consecutive keys of a V fragment, scaled.
__device__ __forceinline__ void value_pairs(uint32_t codes, uint32_t scales, half2v* pr) {
  const half2v a = e4m3_pair<true>(scales, 0), b = e4m3_pair<true>(scales, 1);
  pr[0] = e2m1x2_to_f16<0>(codes) * half2v{a.x, a.x};
  pr[1] = e2m1x2_to_f16<1>(codes) * half2v{a.y, a.y};
  pr[2] = e2m1x2_to_f16<2>(codes) * half2v{b.x, b.x};
  pr[3] = e2m1x2_to_f16<3>(codes) * half2v{b.y, b.y};
}

// The two E2M1 codes of byte `sel` (a constant once unrolled) as fp16.
__device__ __forceinline__ half2v e2m1x2_byte(uint32_t w, int sel) {
  return sel == 0 ? e2m1x2_to_f16<0>(w) : sel == 1 ? e2m1x2_to_f16<1>(w) : sel == 2 ? e2m1x2_to_f16<2>(w) : e2m1x2_to_f16<3>(w);
}

template <int D, int kTiles, bool kWide>
__global__ __launch_bounds__(256, (Stream<D, kTiles>::kOccupancy)) void kv_attention_stream_kernel(KvCache c, KvAttention a,
                                                                                                Cut cut) {
  using T = Stream<D, kTiles>;
  constexpr int kW = T::kKWords, kP = T::kPairs, kS = T::kSWords;
  __shared__ float red_ml[2][T::kWaves][16];
  __shared__ __align__(16) float red_o[T::kWaves][16][D + 4];
  __shared__ __align__(16) uint8_t scales_lds[T::kWaves][2][2][4 * D];       // [wave][pass parity][K, V]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, r = lane & 15;
  const int group = a.q_heads / c.heads;

  const float k_gscale = *c.k_gscale, v_gscale = *c.v_gscale;

  // ---- which segments: one, or a worker's share of all passes
  Item it;
  int todo = 0, pass = 0, tile = 0, worker = 0, len = -1;      // passes left of the share, the sequence's length
  int64_t prefix_at = 0;
  const bool even = blockIdx.x >= cut.prefix_items && cut.workers > 0;
  if (blockIdx.x < cut.prefix_items) {
    const uint32_t ch = blockIdx.x % cut.prefix_chunks, rest = blockIdx.x / cut.prefix_chunks;
    it.row0 = (int)(rest % cut.prefix_tiles) * T::kRows;
    it.kvh = (int)(rest / cut.prefix_tiles);
    it.pages = a.prefix_pages;
    it.key0 = (int)ch * cut.prefix_chunk;
    it.key1 = min(it.key0 + cut.prefix_chunk, a.prefix_len);
    it.q0 = 0;
    it.rows = (int)a.total_q * group;
    it.seq = -1;
    prefix_at = ch;
  } else {
    const int x = (int)(blockIdx.x - cut.prefix_items);
    if (!even) {
      it.seq = x % a.batch;
      tile = x / a.batch;
    } else {
      worker = x;
      int first = 0;
      const Spot spot = spot_of<true>(a, 0, [&](int all) {
        const int total = all * c.heads * cut.own_tiles;
        const int share = share_of(cut, total);
        first = worker * share;
        todo = min(share, total - first);
        if (todo <= 0) return 0;
        tile = first / all;
        return first - tile * all;
      });
      if (todo <= 0) return;
      it.seq = spot.seq;
      len = spot.len;
      pass = first - tile * spot.all - spot.before;
    }
  }

  for (;;) {
    int end_pass = 0, passes = 0;
    if (it.seq >= 0) {
      own_rows_of(a, group, it);
      it.kvh = tile / cut.own_tiles;
      it.row0 = (tile - it.kvh * cut.own_tiles) * T::kRows;
      if (len < 0) len = own_length(a, it.seq);
      passes = passes_of(len);
      end_pass = even ? min(passes, pass + todo) : passes;
      it.key0 = pass * kPass;
      it.key1 = min(end_pass * kPass, len);
    }
    if (it.row0 < it.rows) {
      float4v acc[kTiles][kP][2], sum[kTiles];
      float mx[kTiles];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        mx[m] = -__builtin_inff();
        sum[m] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < kP; ++u) acc[m][u][0] = acc[m][u][1] = float4v{0.f, 0.f, 0.f, 0.f};
      }
      const _Float16 one = (_Float16)1.0f;
      const half8v ones{one, one, one, one, one, one, one, one};

      // past the last row's limit every row is masked (rows of one sequence see more and more)
      const int last_row = min(it.row0 + T::kRows, it.rows) - 1;
      const int key1 = it.seq < 0 ? it.key1 : min(it.key1, own_limit(len, it.q0, it.n, it.q0 + last_row / group));
      const int mask_in_page = (1 << c.ps_log2) - 1;
      const int64_t page_rows = (int64_t)c.heads << c.ps_log2;
      const int64_t head_row = (int64_t)it.kvh << c.ps_log2;
      const int last = it.key1 - 1;
      int zero = 0;
      asm volatile("" : "+v"(zero));                  // keeps the page load a vector load
      // Pages: of the fragments a lane takes K codes from (r / 4) and everything
      // else from (g).  Pages of 64 keys or more hold a whole pass of a wave: with
      // kWide one page number serves it and every address is a scalar base and a
      // lane offset that never changes (48 single tokens, 12 on 4 heads of 64
      // values: 34.9 us, 36.2 the other way; 16 sequences of 32 rows of 128 values
      // 42.2 and 43.0; single tokens on heads of 128 and 60 rows of 256 alike).
      // A fragment past the segment's end takes
      // its last key's page, one outside the pool page 0 (masked).  Page numbers
      // are carried as they are in memory, so that a load in flight is first
      // waited for where it is used (a scalar load would be waited for by the
      // next LDS access).
      struct Pages { int k, v; };
      auto page_of = [&](int key) { return it.pages[min(key, last) >> c.ps_log2]; };
      auto pages_at = [&](int key) {
        if constexpr (kWide) {
          int p;
          const int32_t* at = it.pages + (min(key, last) >> c.ps_log2) + (lane & zero);
          p = *at;
          return Pages{p, p};
        } else {
          return Pages{page_of(key + 16 * (r >> 2)), page_of(key + 16 * g)};
        }
      };
      auto settled = [&](Pages p) {                   // at the use: into a scalar
        if constexpr (kWide) p.k = p.v = __builtin_amdgcn_readfirstlane(p.v);
        return p;
      };
      auto in_pool = [&](int page) { return (uint32_t)page < (uint32_t)c.num_pages; };
      // the cache row the lane offsets below count from: of the pass, or of the
      // lane's fragment
      auto base_row = [&](int key, int frag, int page) {
        const int at = (kWide ? key : key + 16 * frag) & mask_in_page;
        return (int64_t)(in_pool(page) ? page : 0) * page_rows + head_row + at;
      };
      const int fk = kWide ? 16 * (r >> 2) : 0, fg = kWide ? 16 * g : 0;
      const uint32_t k_lane = (fk + (r & 3)) * (D / 2) + g * (D / 8), v_lane = fg * (D / 2) + r * 16;
      const uint32_t s_lane = (fg + r) * (D / 16);
      uint32_t kc[4][kW], vc[kP][4], ksr[kS], vsr[kS];
      auto load_k = [&](int key, Pages p) {
        const uint8_t* b = c.k_codes + base_row(key, r >> 2, p.k) * (D / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_words<kW>(b + (k_lane + i * (4 * D / 2)), kc[i]);
      };
      auto load_v = [&](int key, Pages p) {
        const uint8_t* b = c.v_codes + base_row(key, g, p.v) * (D / 2);
#pragma unroll
        for (int u = 0; u < kP; ++u) load_words<4>(b + (v_lane + u * 256), vc[u]);
      };
      // D/16 bytes a lane: K's of key 16 g + r, and V's from byte r D/16 of fragment g
      auto load_scales = [&](int key, Pages p) {
        const int64_t off = base_row(key, g, p.v) * (D / 16);
        load_words<kS>(c.k_scales + off + s_lane, ksr);
        load_words<kS>(c.v_scales + off + s_lane, vsr);
      };
      auto stage_scales = [&](int key, Pages p, int par) {
        // V bytes of keys that were never written may be NaN, and 0 * NaN is not 0
        const int n = in_pool(p.v) ? it.key1 - (key + 16 * g) : 0;
        if (__any(n < 16)) {
#pragma unroll
          for (int x = 0; x < kS; ++x) {
            const int keep = min(max(n - ((r * (D / 16)) & 15) - 4 * x, 0), 4);
            vsr[x] &= keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
          }
        }
        store_words<kS>(&scales_lds[wave][par][0][lane * (D / 16)], ksr);
        store_words<kS>(&scales_lds[wave][par][1][lane * (D / 16)], vsr);
      };
      constexpr int kStep = 64 * T::kWaves;
      int key = it.key0 + 64 * wave, par = 0;
      // the pass after `key`; at the end the last one again (cache hits): loads
      // under a condition would make every wait below one for all of them
      auto after = [&](int k) { return k + kStep < key1 ? k + kStep : k; };
      if (key < key1) {
      const int k1 = after(key), k2 = after(k1);
      Pages p0 = pages_at(key), p1 = pages_at(k1), p2 = pages_at(k2);       // of this pass, the next, the one after
      uint32_t qw[kTiles][kW * 4];
      int limit[kTiles], limit_min = 0x7FFFFFFF;
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        const int row = it.row0 + 16 * m + r;
        const bool live = row < it.rows;
        const int x = live ? row : 0, t = it.q0 + x / group, h = it.kvh * group + x % group;
        load_words<kW * 4>(reinterpret_cast<const uint8_t*>(a.q + t * a.q_stride + (int64_t)h * D + g * (D / 4)), qw[m]);
        limit[m] = !live ? 0 : it.seq < 0 ? prefix_limit(a, t) : own_limit(len, it.q0, it.n, t);
        limit_min = min(limit_min, live ? limit[m] : 0x7FFFFFFF);
      }
      // in the order of the loop, so that its waits are counted the same
      p0 = settled(p0);
      p1 = settled(p1);
      load_scales(key, p0);
      load_k(key, p0);
      stage_scales(key, p0, 0);
      load_scales(k1, p1);
      load_v(key, p0);
      asm volatile("; first pass requested" ::: "memory");

      // Q: each row scaled by a power of two to a largest magnitude in [2^14,
      // 2^15), then exact in fp16 down to 2^-31 of it; the inverse goes into the
      // score factor.  A row with an infinity or NaN gets a NaN factor.
      half8v qf[kTiles][kW];
      float factor[kTiles];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kW * 4; ++i) top = max(top, bf16x2_absmax_bits(qw[m][i]));
        top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        const int e = (int)(top >> 7);                                // biased exponent of the largest
        const int sh = e == 0 ? 0 : 141 - e;                          // to 2^14, exponent 127 + 14
        // 2^sh in two exact steps (|sh| may pass 127 for tiny rows)
        const float f1 = __uint_as_float((uint32_t)(127 + sh / 2) << 23);
        const float f2 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
#pragma unroll
        for (int s = 0; s < kW; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = qw[m][4 * s + i];
            qf[m][s][2 * i] = (_Float16)(__uint_as_float(v << 16) * f1 * f2);
            qf[m][s][2 * i + 1] = (_Float16)(__uint_as_float(v & 0xFFFF0000u) * f1 * f2);
          }
        const float i1 = __uint_as_float((uint32_t)(127 - sh / 2) << 23);
        const float i2 = __uint_as_float((uint32_t)(127 - (sh - sh / 2)) << 23);
        factor[m] = score_factor(e, a.scale, k_gscale, i1, i2);
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) limit_min = min(limit_min, __shfl_xor(limit_min, o, 64));

      for (; key < key1; key += kStep) {
        const int next = after(key), next2 = after(next);
        // ---- scores
        float4v st[kTiles][4];
        const uint8_t* ks = scales_lds[wave][par][0] + (16 * (r >> 2) + (r & 3)) * (D / 16) + g * (D / 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t sw = load_k_scales<D>(ks + i * (4 * D / 16));
#pragma unroll
          for (int m = 0; m < kTiles; ++m) st[m][i] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < kW; ++s) {
            // two steps share a block scale (bytes of keys that were never
            // written may be NaN: their scores are masked below)
            const half2v pair = e4m3_pair<D == 256>(sw, s >> 2);
            const half8v kf = dequant8_f16(kc[i][s], (s >> 1) & 1 ? half2v{pair.y, pair.y} : half2v{pair.x, pair.x});
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
              st[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[m][s], st[m][i], 0, 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);     // keeps the decoded values of one tile at a time in registers
        }
        p2 = settled(p2);
        stage_scales(next, p1, par ^ 1);
        load_k(next, p1);
        load_scales(next2, p2);
        const bool v_ok = in_pool(p0.v);
        p0 = p1;
        p1 = p2;
        p2 = pages_at(after(next2));
        // ---- softmax weights
        const int k0 = key + 16 * g;
        const bool whole = key + 64 <= min(limit_min, it.key1) && __all(v_ok);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          if (!whole) {
            const int n = v_ok ? min(it.key1, limit[m]) - k0 : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (4 * i + j >= n) st[m][i][j] = -__builtin_inff();
          }
          float top = -__builtin_inff();
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = fmaxf(top, st[m][i][j]);
          top = fmaxf(top, __shfl_xor(top, 16, 64));
          top = fmaxf(top, __shfl_xor(top, 32, 64));
          top *= factor[m];
          if (__any(top > mx[m] + kLag)) {
            const float now = top > mx[m] + kLag ? top : mx[m];
            const float f = exp2_hw(mx[m] - finite_or_zero(now));
            mx[m] = now;
            sum[m][0] *= f;
#pragma unroll
            for (int u = 0; u < kP; ++u) {
              // see the tile kernel: keeps copies of the sums off the usual path
              if constexpr (D == 256) asm volatile("" : "+a"(acc[m][u][0]), "+a"(acc[m][u][1]));
              acc[m][u][0] *= f;
              acc[m][u][1] *= f;
            }
          }
          const float base = kBias - finite_or_zero(mx[m]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) st[m][i][j] = exp2_hw(__builtin_fmaf(st[m][i][j], factor[m], base));
        }
        // ---- weighted values
        const uint8_t* vs = scales_lds[wave][par][1] + g * D + (r >> 3) * 16;
        if constexpr (kTiles == 1) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {                       // 4 keys a step
            half8v even_p, odd_p;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const half2v e = __builtin_convertvector(float2v{st[0][x][j], 0.0f}, half2v);
              const half2v o = __builtin_convertvector(float2v{0.0f, st[0][x][j]}, half2v);
              even_p[2 * j] = e.x; even_p[2 * j + 1] = e.y;
              odd_p[2 * j] = o.x; odd_p[2 * j + 1] = o.y;
            }
            sum[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, even_p, sum[0], 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kP; ++u) {
              half2v pr[4];
              value_pairs(vc[u][x], *reinterpret_cast<const uint32_t*>(vs + u * 32 + 4 * x), pr);
              const half8v vf{pr[0].x, pr[0].y, pr[1].x, pr[1].y, pr[2].x, pr[2].y, pr[3].x, pr[3].y};
              acc[0][u][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, even_p, acc[0][u][0], 0, 0, 0);
              acc[0][u][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, odd_p, acc[0][u][1], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x) {                       // 8 keys a step
            half8v pw[kTiles];
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                const half2v e = __builtin_convertvector(
                    float2v{st[m][2 * x + i / 4][i % 4], st[m][2 * x + i / 4][i % 4 + 1]}, half2v);
                pw[m][i] = e.x; pw[m][i + 1] = e.y;
              }
              sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pw[m], sum[m], 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kP; ++u) {
              half2v pr[8];
              const uint2 sw = *reinterpret_cast<const uint2*>(vs + u * 32 + 8 * x);
              value_pairs(vc[u][2 * x], sw.x, pr);
              value_pairs(vc[u][2 * x + 1], sw.y, pr + 4);
              half8v lo, hi;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                lo[i] = pr[i].x;
                hi[i] = pr[i].y;
              }
#pragma unroll
              for (int m = 0; m < kTiles; ++m) {
                acc[m][u][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, pw[m], acc[m][u][0], 0, 0, 0);
                acc[m][u][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, pw[m], acc[m][u][1], 0, 0, 0);
              }
            }
          }
        }
        load_v(next, p0);
        par ^= 1;
        // without these two marks the compiler merges this load with the first
        // one, into the top of the loop, where nothing hides it
        asm volatile("; next pass requested" ::: "memory");
      }
      }

      // ---- join the waves: lane (g, r) holds row r's values 32 u + 8 g .. + 7
      const bool begun = even && pass > 0, cut_off = even && end_pass < passes;
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        __syncthreads();                       // the previous tile's results are taken
        if (g == 0) {
          red_ml[0][wave][r] = mx[m];
          red_ml[1][wave][r] = sum[m][0];
        }
#pragma unroll
        for (int u = 0; u < kP; ++u) {
          float* dst = &red_o[wave][r][32 * u + 8 * g];
          const float4v e = acc[m][u][0], o = acc[m][u][1];
          *reinterpret_cast<float4v*>(dst) = float4v{e[0], o[0], e[1], o[1]};
          *reinterpret_cast<float4v*>(dst + 4) = float4v{e[2], o[2], e[3], o[3]};
        }
        __syncthreads();
        const int x = threadIdx.x >> 4, piece = threadIdx.x & 15;     // row, D/16 values
        const int row = it.row0 + 16 * m + x;
        if (row < it.rows) {
          float top = -__builtin_inff();
#pragma unroll
          for (int w = 0; w < T::kWaves; ++w) top = fmaxf(top, red_ml[0][w][x]);
          float wt[T::kWaves], lsum = 0.0f;
#pragma unroll
          for (int w = 0; w < T::kWaves; ++w) {
            wt[w] = exp2_hw(red_ml[0][w][x] - finite_or_zero(top));
            lsum += wt[w] * red_ml[1][w][x];
          }
          float o[D / 16];
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < T::kWaves; ++w) o[i] = __builtin_fmaf(wt[w], red_o[w][x][piece * (D / 16) + i], o[i]);
          }
          const int t = it.q0 + row / group, h = it.kvh * group + row % group;
          const int64_t orow = (int64_t)t * a.q_heads + h;
          int64_t at;
          if (it.seq < 0) at = orow * cut.prefix_chunks + prefix_at;
          else if (begun || cut_off) at = cut.slot_at + ((int64_t)worker * 2 + (begun ? 0 : 1)) * cut.own_rows + 16 * m + x;
          else at = a.prefix_len > 0 ? cut.full_at + orow : -1;
          if (at < 0) {
            const float inv = lsum == 0.0f ? 0.0f : v_gscale / lsum;
            uint32_t out[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) out[i] = f32x2_to_bf16x2_rne(o[2 * i] * inv, o[2 * i + 1] * inv);
            uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + piece * (D / 16));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) dst[i] = out[i];
          } else {
            if (piece == 0) *reinterpret_cast<float2*>(cut.part_ml + at * 2) = make_float2(top, lsum);
            float* dst = cut.part_o + at * D + piece * (D / 16);
#pragma unroll
            for (int i = 0; i < D / 16; i += 4)
              *reinterpret_cast<float4v*>(dst + i) = float4v{o[i], o[i + 1], o[i + 2], o[i + 3]};
          }
        }
      }
    }
    if (!even) return;
    todo -= end_pass - pass;
    if (todo <= 0) return;
    pass = 0;
    len = -1;
    if (++it.seq == a.batch) {
      it.seq = 0;
      ++tile;
    }
  }
}

// ---- many rows: decoded tiles in LDS -----------------------------------------
//
// A workgroup takes 32 rows for each of its kWaves waves against blocks of 64
// keys, which are decoded to fp16 once for all of them and staged in LDS
// (two buffers, one barrier a block).  With lane = 32 h + r (the layout of
// v_mfma_f32_32x32x16_f16: operands hold row or column r at k = 8 h .. 8 h + 7,
// results column r at rows 8 (i / 4) + 4 h + i % 4 for i = 0 .. 15):
//   S^T = K Q^T    LDS row x of a 32-key tile holds the key whose number is x
//                  with bits 2 and 3 exchanged, so that lane (h, r) ends up with
//                  query r's scores of keys 16 j + 8 h .. + 7, in order;
//   O^T = V^T P^T  V is staged transposed, [value][key], and those 8 keys are
//                  the lane's contraction slots: P goes from the score registers
//                  to the operand without leaving the lane.
// Rows of LDS are cut into 16-byte units and a row's units are exchanged by its
// number, so that 16 lanes that read or write one unit of 16 rows touch all
// banks.
//
// Bound by the matrix cores and, with them busy, by power.  A chunk of 2 x 2048
// queries, 32 heads on 16 of 128 values, before which 9000 to 16384 keys lie:
// 868 GFLOP in 820 to 893 us, 970 to 1059 TFLOP/s as the card's clock goes; a
// large fp16 library product reaches 1157.  Decoding in the phases between the products, not beside them,
// took 876 us; all waves in one phase at a time, 936; without the tiles in LDS,
// each wave decoding for itself, 1570.  With 64 values the softmax, which costs
// the same for a key, weighs twice as much: 763 TFLOP/s; with 256 the sums leave
// one wave a SIMD, whose softmax stands between its products: 789.
template <int D>
struct Tile {
  // rows a workgroup takes: 8 waves of 32 with two waves to a SIMD, so that one
  // wave's matrix products run under the other's softmax; with D = 256 the
  // sums leave room for one wave to a SIMD
  static constexpr int kWaves = D == 256 ? 4 : 8;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kRows = 32 * kWaves;
  static constexpr int kOccupancy = D == 256 ? 1 : 2;      // waves per SIMD
  static constexpr int kItems = D * 2;                     // 16-byte pieces of K (and of V) codes in a block
  static constexpr int kKBytes = 64 * D * 2;
};
constexpr int kBlockKeys = 64;

// f(0), f(1), ... f(n - 1) with constant arguments.
template <typename F, int... kI>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, kI...>) {
  (f(std::integral_constant<int, kI>{}), ...);
}
template <int kN, typename F>
__device__ __forceinline__ void each(F&& f) {
  each_of(f, std::make_integer_sequence<int, kN>{});
}

template <int D>
__device__ __forceinline__ uint32_t k_unit_at(int row, int unit) {      // byte offset in the K tile
  const int x = D == 64 ? (row >> 1) & 7 : row & 15;
  return row * (D * 2) + ((unit ^ x) << 4);
}
__device__ __forceinline__ uint32_t v_unit_at(int d, int unit) {        // in the V tile
  return d * (kBlockKeys * 2) + ((unit ^ ((d >> 1) & 7)) << 4);
}

template <int D, bool kWide>
__global__ __launch_bounds__(Tile<D>::kThreads, Tile<D>::kOccupancy) void kv_attention_tile_kernel(KvCache c, KvAttention a,
                                                                                                 Cut cut) {
  using T = Tile<D>;
  constexpr int kSteps = D / 16, kDTiles = D / 32;
  // pieces of K and V codes a thread decodes: all threads take K and V pieces,
  // or the first half K and the second half V
  constexpr bool kHalves = T::kItems < T::kThreads;
  constexpr int kPieces = kHalves ? 1 : T::kItems / T::kThreads;
  __shared__ __align__(16) uint8_t tile_k[2][T::kKBytes];
  __shared__ __align__(16) uint8_t tile_v[2][T::kKBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r = lane & 31;
  const int group = a.q_heads / c.heads;
  const float k_gscale = *c.k_gscale, v_gscale = *c.v_gscale;

  Item it;
  int len = 0, chunk;
  if (blockIdx.x < cut.prefix_items) {
    chunk = blockIdx.x % cut.prefix_chunks;
    const int rest = blockIdx.x / cut.prefix_chunks;
    it.row0 = rest % cut.prefix_tiles * T::kRows;
    it.kvh = rest / cut.prefix_tiles;
    it.seq = -1;
    it.pages = a.prefix_pages;
    it.key0 = chunk * cut.prefix_chunk;
    it.key1 = min(it.key0 + cut.prefix_chunk, a.prefix_len);
    it.q0 = 0;
    it.n = it.rows = (int)a.total_q * group;
  } else {
    // the last row tiles of a sequence see the most keys: they go first
    const int x = blockIdx.x - cut.prefix_items;
    chunk = x % cut.own_chunks;
    int rest = x / cut.own_chunks;
    it.kvh = rest % c.heads;
    rest /= c.heads;
    it.seq = rest % a.batch;
    it.row0 = (cut.own_tiles - 1 - rest / a.batch) * T::kRows;
    own_rows_of(a, group, it);
    if (it.row0 >= it.rows) return;
    len = own_length(a, it.seq);
    it.key0 = chunk * cut.own_chunk;
    if (chunk > 0 && it.key0 >= len) return;
    const int last_row = min(it.row0 + T::kRows, it.rows) - 1;
    it.key1 = min(it.key0 + cut.own_chunk, own_limit(len, it.q0, it.n, it.q0 + last_row / group));
  }

  // Q, scaled as in the streaming kernel
  half8v qf[kSteps];
  float factor;
  int limit, limit_min;
  {
    const int row = it.row0 + 32 * wave + r;
    const bool live = row < it.rows;
    const int x = live ? row : 0, t = it.q0 + x / group, hd = it.kvh * group + x % group;
    uint32_t w[kSteps * 4];
    const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q + t * a.q_stride + (int64_t)hd * D + 8 * h);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) load_words<4>(src + 32 * s, w + 4 * s);
    limit = !live ? 0 : it.seq < 0 ? prefix_limit(a, t) : own_limit(len, it.q0, it.n, t);
    limit_min = live ? limit : 0x7FFFFFFF;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kSteps * 4; ++i) top = max(top, bf16x2_absmax_bits(w[i]));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    const int e = (int)(top >> 7), sh = e == 0 ? 0 : 141 - e;
    const float f1 = __uint_as_float((uint32_t)(127 + sh / 2) << 23);
    const float f2 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = w[4 * s + i];
        qf[s][2 * i] = (_Float16)(__uint_as_float(v << 16) * f1 * f2);
        qf[s][2 * i + 1] = (_Float16)(__uint_as_float(v & 0xFFFF0000u) * f1 * f2);
      }
    const float i1 = __uint_as_float((uint32_t)(127 - sh / 2) << 23);
    const float i2 = __uint_as_float((uint32_t)(127 - (sh - sh / 2)) << 23);
    factor = score_factor(e, a.scale, k_gscale, i1, i2);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) limit_min = min(limit_min, __shfl_xor(limit_min, o, 64));
  limit_min = __builtin_amdgcn_readfirstlane(limit_min);

  float16v acc[kDTiles];
  float mx = -__builtin_inff(), sum = 0.0f;
#pragma unroll
  for (int u = 0; u < kDTiles; ++u) acc[u] = float16v{};

  // ---- the pieces of a block this thread decodes: K piece x is 32 values of key
  // x / (D/32), V piece x the value pair x % (D/2) of fragment x / (D/2)
  const int slot = kHalves ? wave & (T::kWaves / 2 - 1) : wave, piece0 = slot * 64 + lane;
  const bool first_half = wave < T::kWaves / 2, busy = slot * 64 < T::kItems;
  const int mask_in_page = (1 << c.ps_log2) - 1;
  const int64_t page_rows = (int64_t)c.heads << c.ps_log2, head_row = (int64_t)it.kvh << c.ps_log2;
  const int last = it.key1 - 1;
  constexpr int kKPieces = D / 32, kVPieces = D / 2;        // of a key; of a fragment
  constexpr int kV = kHalves ? 0 : 1;                       // where V's pieces are kept
  struct Raw {
    uint32_t codes[kV + 1][kPieces][4], scales[kV + 1][kPieces][4];
  };
  int zero = 0;
  asm volatile("" : "+v"(zero));                      // keeps the page loads vector loads
  auto page_of = [&](int key) __attribute__((always_inline)) {
    return it.pages[(min(key, last) >> c.ps_log2) + (kWide ? lane & zero : 0)];
  };
  auto in_pool = [&](int page) __attribute__((always_inline)) { return (uint32_t)page < (uint32_t)c.num_pages; };
  // Page numbers of a block as they come from memory: of the key each piece
  // begins in, and of key number `lane`; with kWide (pages of 64 keys or more)
  // one number is all of them (833 against 853 us for the chunk above, 1106
  // against 1196 with 256 values).
  struct PageLoad {
    int k[kPieces], v[kPieces], mine;
  };
  auto pages_at = [&](int key) __attribute__((always_inline)) {
    PageLoad p;
    p.mine = page_of(kWide ? key : key + lane);
    if constexpr (!kWide) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int x = piece0 + i * T::kThreads;
        p.k[i] = page_of(key + (kHalves && !first_half ? 16 * (x / kVPieces) : x / kKPieces));
        p.v[i] = kHalves ? p.k[i] : page_of(key + 16 * (x / kVPieces));
      }
    }
    return p;
  };
  // The same where they are first used, and which of the 64 keys have a page in
  // the pool.  From D = 128 on a wave's piece lies within a fragment: scalars.
  struct PageSet {
    int k[kPieces], v[kPieces];
    uint64_t pool;
  };
  auto settled = [&](const PageLoad& p) __attribute__((always_inline)) {
    PageSet s;
    const int one = kWide ? __builtin_amdgcn_readfirstlane(p.mine) : 0;
    s.pool = kWide ? (in_pool(one) ? ~0ull : 0ull) : __ballot(in_pool(p.mine));
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      s.k[i] = kWide ? one : D >= 128 ? __builtin_amdgcn_readfirstlane(p.k[i]) : p.k[i];
      s.v[i] = kWide ? one : D >= 128 ? __builtin_amdgcn_readfirstlane(p.v[i]) : p.v[i];
    }
    return s;
  };
  // first row of the block (kWide) or of the 16 keys at `at` in it; a page
  // outside the pool counts as page 0
  auto row_of = [&](int key, int at, int page) __attribute__((always_inline)) {
    return (int64_t)(in_pool(page) ? page : 0) * page_rows + head_row + ((kWide ? key : key + at) & mask_in_page);
  };
  auto load_k = [&](int key, const PageSet& p, Raw& raw) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int x = piece0 + i * T::kThreads, n = x / kKPieces, part = x % kKPieces, extra = kWide ? n : 0;
      const int64_t row = row_of(key, n, p.k[i]);
      load_words<4>(c.k_codes + row * (D / 2) + (uint32_t)(extra * (D / 2) + part * 16), raw.codes[0][i]);
      raw.scales[0][i][0] = *reinterpret_cast<const uint16_t*>(c.k_scales + row * (D / 16) +
                                                               (uint32_t)(extra * (D / 16) + part * 2));
    }
  };
  auto load_v = [&](int key, const PageSet& p, Raw& raw) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int x = piece0 + i * T::kThreads, n = 16 * (x / kVPieces), pair = x % kVPieces, extra = kWide ? n : 0;
      const int64_t row = row_of(key, n, p.v[i]);
      load_words<4>(c.v_codes + row * (D / 2) + (uint32_t)(extra * (D / 2) + pair * 16), raw.codes[kV][i]);
      load_words<4>(c.v_scales + row * (D / 16) + (uint32_t)(extra * (D / 16) + (pair >> 3) * 16), raw.scales[kV][i]);
    }
  };
  // V scale bytes of keys that were never written may be NaN, and 0 * NaN is
  // not 0: those past the end and of pages outside the pool become 0
  auto trim_v = [&](int key, const PageSet& p, Raw& raw) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int frag = (piece0 + i * T::kThreads) / kVPieces;
      const int n = in_pool(p.v[i]) ? it.key1 - (key + 16 * frag) : 0;
      if (__any(n < 16)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int keep = min(max(n - 4 * j, 0), 4);
          raw.scales[kV][i][j] &= keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
        }
      }
    }
  };
  // Decoding in kMicro small steps a piece, to be laid between matrix products:
  // K, step 4 j + y turns byte y of dword j into two values, the last one of a
  // dword stores its 16 bytes; V, steps of word w pair up its nibbles by value,
  // convert the even and the odd value's 4 keys, and store every 8 keys.
  constexpr int kMicro = 16;
  half8v kval, vval[2];
  uint32_t ve, vo;
  half2v vsa, vsb;
  auto k_micro = [&](const Raw& raw, int buf, int step) __attribute__((always_inline)) {
    const int i = step / kMicro, j = step % kMicro / 4, y = step % 4;
    const half2v sc = e4m3_pair<false>(raw.scales[0][i][0], 0);
    const half2v v = e2m1x2_byte(raw.codes[0][i][j], y) * (j < 2 ? half2v{sc.x, sc.x} : half2v{sc.y, sc.y});
    kval[2 * y] = v.x;
    kval[2 * y + 1] = v.y;
    if (y == 3) {
      const int x = piece0 + i * T::kThreads, part = x % kKPieces, n = x / kKPieces;
      const int row = (n & ~12) | ((n & 4) << 1) | ((n & 8) >> 1);
      *reinterpret_cast<half8v*>(&tile_k[buf][k_unit_at<D>(row, 4 * part + j)]) = kval;
    }
  };
  auto v_micro = [&](const Raw& raw, int buf, int step) __attribute__((always_inline)) {
    const int i = step / kMicro, w = step % kMicro / 4, y = step % 4, half_at = 4 * (w & 1);
    if (y == 0) {
      const uint32_t codes = raw.codes[kV][i][w];
      ve = (codes & 0x000F000Fu) | ((codes >> 4) & 0x00F000F0u);       // even value: keys (0, 1), (2, 3) in bytes 0, 2
      vo = (codes & 0xF000F000u) | ((codes << 4) & 0x0F000F00u);       // odd value: in bytes 1, 3
      vsa = e4m3_pair<true>(raw.scales[kV][i][w], 0);
      vsb = e4m3_pair<true>(raw.scales[kV][i][w], 1);
    } else if (y < 3) {
      const uint32_t c4 = y == 1 ? ve : vo;
      const half2v a2 = e2m1x2_byte(c4, y - 1) * vsa, b2 = e2m1x2_byte(c4, y + 1) * vsb;
      vval[y - 1][half_at] = a2.x;
      vval[y - 1][half_at + 1] = a2.y;
      vval[y - 1][half_at + 2] = b2.x;
      vval[y - 1][half_at + 3] = b2.y;
    } else if (w & 1) {
      const int x = piece0 + i * T::kThreads, pair = x % kVPieces, frag = x / kVPieces;
      *reinterpret_cast<half8v*>(&tile_v[buf][v_unit_at(2 * pair, 2 * frag + w / 2)]) = vval[0];
      *reinterpret_cast<half8v*>(&tile_v[buf][v_unit_at(2 * pair + 1, 2 * frag + w / 2)]) = vval[1];
    }
  };
  auto stage_k = [&](const Raw& raw, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kMicro * kPieces; ++i) k_micro(raw, buf, i);
  };
  auto stage_v = [&](const Raw& raw, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kMicro * kPieces; ++i) v_micro(raw, buf, i);
  };

  float16v st[2];
  half8v pw[4];
  auto scores = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      st[kt] = float16v{};
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        st[kt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            *reinterpret_cast<const half8v*>(&tile_k[buf][k_unit_at<D>(32 * kt + r, 2 * s + h)]), qf[s], st[kt], 0, 0, 0);
    }
  };
  auto weights = [&](int key, uint64_t pool) __attribute__((always_inline)) {
    if (key + kBlockKeys > min(limit_min, it.key1) || pool != ~0ull) {
      const int n = min(it.key1, limit) - key;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = 32 * kt + 16 * (i / 8) + 8 * h + i % 8;
          if (x >= n || !((pool >> x) & 1)) st[kt][i] = -__builtin_inff();
        }
    }
    // four chains each: one wave alone does not hide a chain's latency
    float part[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) part[x] = fmaxf(st[x / 2][8 * (x & 1)], st[x / 2][8 * (x & 1) + 1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        part[x] = fmaxf(fmaxf(part[x], st[x / 2][8 * (x & 1) + i]), st[x / 2][8 * (x & 1) + i + 1]);
    float top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * factor;
    if (__any(top > mx + kLag)) {
      const float now = top > mx + kLag ? top : mx;
      const float f = exp2_hw(mx - finite_or_zero(now));
      mx = now;
      sum *= f;
#pragma unroll
      for (int u = 0; u < kDTiles; ++u) {
        // with 256 values the sums lie in the accumulation registers; without
        // the mark they are copied out before the branch, in every block (2 x
        // 2048 queries, 16 heads on 4: 1242 us, 1101 with it)
        if constexpr (D == 256) asm volatile("" : "+a"(acc[u]));
        acc[u] *= f;
      }
    }
    const float base = kBias - finite_or_zero(mx);
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) st[kt][i] = exp2_hw(__builtin_fmaf(st[kt][i], factor, base));
    float add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; i += 2)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const half2v e =
            __builtin_convertvector(float2v{st[x / 2][8 * (x & 1) + i], st[x / 2][8 * (x & 1) + i + 1]}, half2v);
        pw[x][i] = e.x;
        pw[x][i + 1] = e.y;
        add[x] = __builtin_amdgcn_fdot2(e, half2v{(_Float16)1.0f, (_Float16)1.0f}, add[x], false);
      }
    sum += (add[0] + add[1]) + (add[2] + add[3]);
  };
  auto values = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int u = 0; u < kDTiles; ++u)
        acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            *reinterpret_cast<const half8v*>(&tile_v[buf][v_unit_at(32 * u + r, 2 * x + h)]), pw[x], acc[u], 0, 0, 0);
  };
  // end of a phase: nothing is moved across
  auto meet = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    wait_lgkm0();
    barrier_nofence();
    __builtin_amdgcn_sched_barrier(0);
  };

  // A block is a vector phase -- its softmax weights -- and a matrix phase: the
  // products of its weights with V, the next block's scores, and between the
  // products the decoding of blocks to come.  The second half of the waves runs
  // one phase behind the first, so that each SIMD always has one wave in
  // either; the first half decodes K, the second V:
  //   slot 2 j      first: products of j - 1, scores of j, K of j + 1   second: weights of j - 1
  //   slot 2 j + 1  first: weights of j     second: products of j - 1, scores of j, V of j
  // K of j + 1 replaces K of j - 1, V of j that of j - 2, both last read in slot
  // 2 j - 1.
  auto walk = [&](auto stages_k, auto stages_v, auto behind) __attribute__((always_inline)) {
    constexpr bool kStK = decltype(stages_k)::value, kStV = decltype(stages_v)::value, kBehind = decltype(behind)::value;
    auto after = [&](int k) __attribute__((always_inline)) { return k + kBlockKeys < it.key1 ? k + kBlockKeys : k; };
    int key = it.key0, k1 = after(key), k2 = after(k1), k3 = after(k2), buf = 0;
    PageSet p0 = settled(pages_at(key)), p1 = settled(pages_at(k1)), p2 = settled(pages_at(k2)), p3;
    PageLoad coming = pages_at(k3);
    Raw raw;
    if constexpr (kStK) {
      load_k(key, p0, raw);
      stage_k(raw, 0);
      load_k(k1, p1, raw);
    }
    if constexpr (kStV) load_v(key, p0, raw);
    meet();
    if constexpr (kBehind) meet();
    scores(0);
    if constexpr (kStK) {
      stage_k(raw, 1);
      load_k(k2, p2, raw);
    }
    if constexpr (kStV) {
      trim_v(key, p0, raw);
      stage_v(raw, 0);
      load_v(k1, p1, raw);
    }
    meet();
    for (; key + kBlockKeys < it.key1; buf ^= 1) {
      weights(key, p0.pool);
      if constexpr (kStV) trim_v(k1, p1, raw);
      meet();
      asm volatile("" : "+v"(coming.mine));              // waited for here, not where its load was issued
      p3 = settled(coming);
      // Products of the weights with V, then the scores of the next block.
      // Operands come from LDS kAhead products ahead (left to itself the
      // scheduler waits for each right before its product), the decoding lies
      // in between, and the order is kept as written.
      constexpr int kAhead = 6, kVProducts = 4 * kDTiles, kProducts = kVProducts + 2 * kSteps;
      constexpr int kWork = kMicro * kPieces;
      half8v op[kAhead + 1];
      auto fetch = [&](int i) __attribute__((always_inline)) {
        op[i % (kAhead + 1)] =
            i < kVProducts
                ? *reinterpret_cast<const half8v*>(&tile_v[buf][v_unit_at(32 * (i % kDTiles) + r, 2 * (i / kDTiles) + h)])
                : *reinterpret_cast<const half8v*>(&tile_k[buf ^ 1][k_unit_at<D>(
                      32 * ((i - kVProducts) / kSteps) + r, 2 * ((i - kVProducts) % kSteps) + h)]);
      };
      // the codes to decode were requested a block ago; the next ones now
      const Raw now = raw;
      if constexpr (kStK) load_k(k3, p3, raw);
      if constexpr (kStV) load_v(k2, p2, raw);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      each<kAhead>([&](auto i) __attribute__((always_inline)) { fetch(i); });
      each<kProducts>([&](auto index) __attribute__((always_inline)) {
        constexpr int i = decltype(index)::value;
        if constexpr (i + kAhead < kProducts) fetch(i + kAhead);
        const half8v operand = op[i % (kAhead + 1)];
        if constexpr (i < kVProducts) {
          float16v& sums = acc[i % kDTiles];
          sums = __builtin_amdgcn_mfma_f32_32x32x16_f16(operand, pw[i / kDTiles], sums, 0, 0, 0);
        } else {
          constexpr int x = (i - kVProducts) % kSteps;
          float16v& score = st[(i - kVProducts) / kSteps];
          if constexpr (x == 0) score = float16v{};
          score = __builtin_amdgcn_mfma_f32_32x32x16_f16(operand, qf[x], score, 0, 0, 0);
        }
        each<kWork>([&](auto step) __attribute__((always_inline)) {
          constexpr int w = decltype(step)::value;
          if constexpr (w >= i * kWork / kProducts && w < (i + 1) * kWork / kProducts) {
            if constexpr (kStK) k_micro(now, buf, w);
            if constexpr (kStV) v_micro(now, buf ^ 1, w);
          }
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      __builtin_amdgcn_s_setprio(0);
      key = k1;
      k1 = k2;
      k2 = k3;
      k3 = after(k3);
      p0 = p1;
      p1 = p2;
      p2 = p3;
      coming = pages_at(k3);
      meet();
    }
    weights(key, p0.pool);
    meet();
    values(buf);
    if constexpr (kHalves && !kBehind) meet();
  };
  if (it.key0 < it.key1) {
    using Yes = std::true_type;
    using No = std::false_type;
    if constexpr (!kHalves) walk(Yes{}, Yes{}, No{});
    else if (first_half && busy) walk(Yes{}, No{}, No{});
    else if (busy) walk(No{}, Yes{}, Yes{});
    else if constexpr (T::kItems < T::kThreads / 2) {       // waves without a piece (D = 64)
      if (first_half) walk(No{}, No{}, No{});
      else walk(No{}, No{}, Yes{});
    }
  }

  // ---- results: lane (h, r) holds row r's values 32 u + 8 (i / 4) + 4 h + i % 4
  const int row = it.row0 + 32 * wave + r;
  const float l = sum + __shfl_xor(sum, 32, 64);
  if (row >= it.rows) return;
  const int64_t orow = (int64_t)(it.q0 + row / group) * a.q_heads + it.kvh * group + row % group;
  int64_t at = -1;
  if (it.seq < 0) at = orow * cut.prefix_chunks + chunk;
  else if (a.prefix_len > 0 || cut.own_chunks > 1) at = cut.full_at + orow * cut.own_chunks + chunk;
  if (at < 0) {
    const float inv = l == 0.0f ? 0.0f : v_gscale / l;
#pragma unroll
    for (int u = 0; u < kDTiles; ++u)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint2*>(a.out + orow * D + 32 * u + 2 * i + 4 * h) =
            make_uint2(f32x2_to_bf16x2_rne(acc[u][i] * inv, acc[u][i + 1] * inv),
                       f32x2_to_bf16x2_rne(acc[u][i + 2] * inv, acc[u][i + 3] * inv));
  } else {
    if (h == 0) *reinterpret_cast<float2*>(cut.part_ml + 2 * at) = make_float2(mx, l);
#pragma unroll
    for (int u = 0; u < kDTiles; ++u)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4v*>(cut.part_o + at * D + 32 * u + 2 * i + 4 * h) =
            float4v{acc[u][i], acc[u][i + 1], acc[u][i + 2], acc[u][i + 3]};
  }
}

// ---- join of partial results --------------------------------------------------

// kRowWaves waves a row; D/4 lanes take a part at a time, four values each, so a
// wave has 256/D parts under way, and loads four of each before it weights them
// by a running maximum: the parts' loads depend on nothing but the lengths.
// Bound by latency: 3 us for 32 rows of 5 parts, 8 for 4096 rows of 18.
template <int D, int kRowWaves>
__global__ __launch_bounds__(256) void kv_attention_join_kernel(KvCache c, KvAttention a, Cut cut) {
  constexpr int kLanes = D / 4, kSubs = 64 / kLanes, kStep = kSubs * kRowWaves, kRows = 4 / kRowWaves;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * kRows + wave / kRowWaves;
  const bool live = row < a.total_q * a.q_heads;
  const int t = live ? (int)(row / a.q_heads) : 0, h = live ? (int)(row - (int64_t)t * a.q_heads) : 0;
  const int b = sequence_of(a, t), group = a.q_heads / c.heads;
  // a query past max_q_len of its sequence, or behind the last one, has no segments
  const int q0 = a.q_starts ? max(0, a.q_starts[b]) : b, q1 = a.q_starts ? a.q_starts[b + 1] : b + 1;
  const int64_t query = (int64_t)t - q0;
  const bool taken = live && t >= q0 && t < q1 && query < a.max_q_len;
  // the row's parts: prefix_chunks of the prefix, then its own
  int own = 1;
  int64_t own_at = cut.full_at + row * cut.own_chunks, own_step = 1, first_off = 0;
  if (cut.own_chunks > 1) own = max(1, (own_length(a, b) + cut.own_chunk - 1) / cut.own_chunk);
  if (cut.workers > 0) {
    const Spot spot = spot_of<false>(a, b, [](int) { return 0; });
    const int share = share_of(cut, spot.all * c.heads * cut.own_tiles);
    if (taken) {
      const int local = (int)query * group + h % group;
      const int s0 = ((h / group) * cut.own_tiles + local / cut.own_rows) * spot.all + spot.before;
      const int first = s0 / share;
      own = (s0 + passes_of(spot.len) - 1) / share - first + 1;
      if (own > 1) {
        // the first part is in its worker's slot 1, the others in slot 0
        own_at = cut.slot_at + (int64_t)first * 2 * cut.own_rows + local % cut.own_rows;
        own_step = 2 * cut.own_rows;
        first_off = cut.own_rows;
      }
    }
  }
  const bool joined = taken && (own > 1 || cut.own_chunks > 1 || cut.prefix_chunks > 0);    // else its workgroup wrote the output
  const int parts = joined ? cut.prefix_chunks + own : 0;
  auto index = [&](int p) {
    if (p < cut.prefix_chunks) return row * cut.prefix_chunks + p;
    const int i = p - cut.prefix_chunks;
    return own_at + i * own_step + (i == 0 ? first_off : 0);
  };
  float m = -__builtin_inff(), l = 0.0f;
  float4v o{0.0f, 0.0f, 0.0f, 0.0f};
  // takes weights relative to m2 in, all rescaled to the larger maximum
  auto add = [&](float m2, float l2, float4v o2) {
    const float top = fmaxf(m, m2), at = finite_or_zero(top), w = exp2_hw(m - at), w2 = exp2_hw(m2 - at);
    l = __builtin_fmaf(w2, l2, w * l);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(w2, o2[i], w * o[i]);
    m = top;
  };
  for (int p = wave % kRowWaves * kSubs + lane / kLanes; p < parts; p += 4 * kStep) {
    float2 ml[4];
    float4v x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = index(min(p + i * kStep, parts - 1));
      ml[i] = *reinterpret_cast<const float2*>(cut.part_ml + 2 * at);
      x[i] = *reinterpret_cast<const float4v*>(cut.part_o + at * D + 4 * (lane % kLanes));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p + i * kStep < parts) add(ml[i].x, ml[i].y, x[i]);
  }
#pragma unroll
  for (int s = kLanes; s < 64; s <<= 1) {
    float4v x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __shfl_xor(o[i], s, 64);
    add(__shfl_xor(m, s, 64), __shfl_xor(l, s, 64), x);
  }
  if constexpr (kRowWaves > 1) {
    __shared__ float2 ml_s[kRowWaves];
    __shared__ float4v o_s[kRowWaves][kLanes];
    if (lane == 0) ml_s[wave] = make_float2(m, l);
    if (lane < kLanes) o_s[wave][lane] = o;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 1; i < kRowWaves; ++i) add(ml_s[i].x, ml_s[i].y, o_s[i][lane % kLanes]);
  }
  if (!joined || lane >= kLanes) return;
  const float inv = l == 0.0f ? 0.0f : *c.v_gscale / l;
  *reinterpret_cast<uint2*>(a.out + row * D + 4 * lane) =
      make_uint2(f32x2_to_bf16x2_rne(o[0] * inv, o[1] * inv), f32x2_to_bf16x2_rne(o[2] * inv, o[3] * inv));
}

// ---- host -------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int tile_rows(int d) { return d == 64 ? Tile<64>::kRows : d == 128 ? Tile<128>::kRows : Tile<256>::kRows; }

// Row tiles (of 16) a streaming workgroup takes for `rows` rows a head, with
// `passes` passes for all heads together; 0: the tile kernel takes them.
//   One while all passes of all tiles are at most eight for every compute unit:
//   the call waits for latencies then, and more workgroups beat fewer reads (24
//   rows of 256 values, 4 heads: 12.7 against 24.5 us with two tiles at 1503
//   keys, 21 against 32 at 20000, but 74 against 61 at 16 x 4000 to 16000) and beat
//   the tile kernel (4 heads of 128 values: 256 rows x 3000 keys 15 against 30
//   us, 2048 x 600 15 against 25, 512 x 3000 24 against 27; past the limit 1024
//   x 3000 32 and 32, 256 x 20000 37 against 34).
//   Otherwise two, while they cost less than the tile kernel, which takes the
//   same time for each of its tiles whether full or not: that of 5.75 pairs of
//   row tiles (of 3.5 with 256 values, where it has 128 rows for 256).
//   Sequences of 8000 to 16000 keys, every one with this many rows a head, in
//   us, two row tiles against the tile kernel:
//                           rows  32      96      128     160     192     256     288
//     24 on 8 heads of  64   61/255 141/262 173/259 221/264 252/272 318/279 372/495
//     24 on 8 heads of 128   90/326 229/346 272/354 355/364 391/373 494/392 590/658
//     4 on 8 heads of 128    31/68   51/74   61/76   71/78   80/80  102/84  111/129
//     24 on 4 heads of 256   95/273 232/290 279/296 372/527 404/523 581/533 617/848
//   (64 values at 192 rows and 256 at 128 would do a few percent better the other way).
int stream_tiles(int64_t rows, int d, int64_t passes) {
  if (rows <= 16 || passes * ceil_div(rows, 16) <= 8 * device_cus()) return 1;
  return 4 * ceil_div(rows, 32) < (d < 256 ? 23 : 14) * ceil_div(rows, tile_rows(d)) ? 2 : 0;
}

// Workgroups the streaming kernel keeps on the card at once.
int stream_workers(int d, int mt) {
  const int per_cu = d == 64    ? (mt == 1 ? Stream<64, 1>::kOccupancy : Stream<64, 2>::kOccupancy)
                     : d == 128 ? (mt == 1 ? Stream<128, 1>::kOccupancy : Stream<128, 2>::kOccupancy)
                                : (mt == 1 ? Stream<256, 1>::kOccupancy : Stream<256, 2>::kOccupancy);
  return per_cu * device_cus();
}

// Chunks of `keys` keys for `base` tile workgroups a chunk, by the rounds of the
// card (a workgroup a compute unit) and the keys a workgroup takes, of which its
// start and end and its share of the join cost some 512: one round of 2048 keys
// takes 108 us and two of half that 126 (512 rows x 8 heads x 32728 keys), but
// 24 x 8 tiles of 64 values in four chunks, three full rounds, 283 against 305 in
// a round three quarters full, 24 x 4 of 256 values 296 against 343 (of 128
// values both 392).  With 64, 128 and 256 values anything from 256 to 2048 in
// the place of 512 measures alike; 64 cuts too finely (256 rows x 8 heads x
// 30000 keys of 64 values: 189 us, 167).  None shorter than 256 keys (512: 36
// against 32 us for 1024 rows x 4 heads x 3000 keys).
void cut_tiles(int64_t keys, int64_t base, int& chunks, int& chunk) {
  const int64_t cus = device_cus(), most = std::max<int64_t>(1, keys / 256);
  int64_t want = 1, least = INT64_MAX;
  for (int64_t rounds = 1; rounds <= 4; ++rounds) {
    const int64_t n = std::min(std::max<int64_t>(1, rounds * cus / std::max<int64_t>(1, base)), most);
    const int64_t cost = ceil_div(base * n, cus) * (ceil_div(keys, n) + 512);
    if (cost < least) {
      least = cost;
      want = n;
    }
  }
  chunk = (int)(ceil_div(ceil_div(std::max<int64_t>(keys, 1), want), kBlockKeys) * kBlockKeys);
  chunks = (int)std::max<int64_t>(1, ceil_div(keys, chunk));
}

struct Plan {
  Cut cut;
  int prefix_mt, own_mt;               // row tiles of 16 of the streaming kernel, 0: the tile kernel
  int64_t prefix_items, own_items;
  int64_t parts;                       // partial results in the workspace
};

Plan make_plan(const KvCache& c, const KvAttention& a) {
  Plan p{};
  const int group = a.q_heads / c.heads, d = c.head_dim;
  const int64_t own_rows = (int64_t)a.max_q_len * group, pre_rows = a.total_q * group, rows = a.total_q * a.q_heads;
  p.cut.own_chunks = 1;
  p.own_mt = stream_tiles(own_rows, d, (int64_t)a.batch * c.heads * ceil_div(a.max_kv_len, kPass));
  if (p.own_mt == 0) {
    p.cut.own_rows = tile_rows(d);
    p.cut.own_tiles = (int)ceil_div(own_rows, p.cut.own_rows);
    const int64_t base = (int64_t)a.batch * c.heads * p.cut.own_tiles;
    cut_tiles(a.max_kv_len, base, p.cut.own_chunks, p.cut.own_chunk);
    p.own_items = base * p.cut.own_chunks;
  } else {
    p.cut.own_rows = 16 * p.own_mt;
    p.cut.own_tiles = (int)ceil_div(own_rows, p.cut.own_rows);
    p.own_items = (int64_t)a.batch * c.heads * p.cut.own_tiles;
    // Segments stay whole unless dealing their passes out evenly shortens the
    // longest place's share by more than three passes, which is what the join
    // and the workers' search for their sequences cost: 64 sequences of 1 to
    // 1024 keys on 8 heads of 128 take 17.3 us whole and 24.5 in shares, but one
    // of 1025 on 16 heads 12.7 and 10.1.
    const int64_t longest = ceil_div(a.max_kv_len, kPass), places = stream_workers(d, p.own_mt), all = p.own_items * longest;
    if (longest * ceil_div(p.own_items, places) > ceil_div(all, places) + 3) {
      p.cut.workers = (int)std::min(places, all);
      p.own_items = p.cut.workers;
    }
  }
  if (a.prefix_len > 0) {
    int64_t base;
    p.prefix_mt = stream_tiles(pre_rows, d, c.heads * ceil_div(a.prefix_len, kPass));
    if (p.prefix_mt == 0) {
      p.cut.prefix_tiles = (int)ceil_div(pre_rows, tile_rows(d));
      base = (int64_t)c.heads * p.cut.prefix_tiles;
      cut_tiles(a.prefix_len, base, p.cut.prefix_chunks, p.cut.prefix_chunk);
    } else {
      // chunks enough for one workgroup on every place, each a pass at least
      p.cut.prefix_tiles = (int)ceil_div(pre_rows, 16 * p.prefix_mt);
      base = (int64_t)c.heads * p.cut.prefix_tiles;
      const int64_t passes = ceil_div(a.prefix_len, kPass);
      const int64_t want = std::min(passes, std::max<int64_t>(1, stream_workers(d, p.prefix_mt) / base));
      p.cut.prefix_chunk = (int)(ceil_div(passes, want) * kPass);
      p.cut.prefix_chunks = (int)ceil_div(a.prefix_len, p.cut.prefix_chunk);
    }
    p.prefix_items = base * p.cut.prefix_chunks;
  }
  p.cut.full_at = rows * p.cut.prefix_chunks;
  p.cut.slot_at = p.cut.full_at + (a.prefix_len > 0 || p.cut.own_chunks > 1 ? rows * p.cut.own_chunks : 0);
  p.parts = p.cut.slot_at + (int64_t)p.cut.workers * 2 * p.cut.own_rows;
  return p;
}

template <int D>
void run_stream(int mt, int64_t items, const KvCache& c, const KvAttention& a, const Cut& cut, hipStream_t st) {
  const dim3 grid((uint32_t)items);
  const bool wide = c.ps_log2 >= 6;
  if (mt == 1 && wide) kv_attention_stream_kernel<D, 1, true><<<grid, 256, 0, st>>>(c, a, cut);
  else if (mt == 1) kv_attention_stream_kernel<D, 1, false><<<grid, 256, 0, st>>>(c, a, cut);
  else if (wide) kv_attention_stream_kernel<D, 2, true><<<grid, 256, 0, st>>>(c, a, cut);
  else kv_attention_stream_kernel<D, 2, false><<<grid, 256, 0, st>>>(c, a, cut);
}

// One launch of the kernel that mt names (see Plan).
template <int D>
void run_items(int mt, int64_t prefix_items, int64_t own_items, const KvCache& c, const KvAttention& a, Cut cut,
               hipStream_t st) {
  cut.prefix_items = (uint32_t)prefix_items;
  if (mt > 0) run_stream<D>(mt, prefix_items + own_items, c, a, cut, st);
  else if (c.ps_log2 >= 6)
    kv_attention_tile_kernel<D, true><<<dim3((uint32_t)(prefix_items + own_items)), Tile<D>::kThreads, 0, st>>>(c, a, cut);
  else
    kv_attention_tile_kernel<D, false><<<dim3((uint32_t)(prefix_items + own_items)), Tile<D>::kThreads, 0, st>>>(c, a, cut);
}

template <int D>
void run_attention(const KvCache& c, const KvAttention& a, const Plan& p, hipStream_t st) {
  if (p.prefix_items > 0 && p.prefix_mt != p.own_mt) {
    run_items<D>(p.prefix_mt, p.prefix_items, 0, c, a, p.cut, st);
    run_items<D>(p.own_mt, 0, p.own_items, c, a, p.cut, st);
  } else {
    run_items<D>(p.own_mt, p.prefix_items, p.own_items, c, a, p.cut, st);
  }
  if (p.parts == 0) return;
  // one wave a row, or four where few rows may have more parts than a wave loads
  // at once: 64 rows of 96 parts of 128 values take 125 against 133 us for the
  // call, 96 rows of 7 parts of 256 values 12.4 against 13.0, 32 of 79 parts of
  // 64 values 13.0 against 14.7, but 32 rows of 5 parts of 128 values 10.3
  // against 10.0, 32 of 16 parts of 64 values 9.4 against 9.3, and 4096 rows of
  // 18 parts 12.0 against 8.3 us in this kernel
  const int64_t own_parts = std::max<int64_t>(p.cut.own_chunks, p.cut.workers / ((int64_t)a.batch * c.heads * p.cut.own_tiles) + 1);
  const int64_t rows = a.total_q * a.q_heads;
  if (rows >= 1024 || p.cut.prefix_chunks + own_parts <= 4 * (256 / D))
    kv_attention_join_kernel<D, 1><<<dim3((uint32_t)ceil_div(rows, 4)), 256, 0, st>>>(c, a, p.cut);
  else
    kv_attention_join_kernel<D, 4><<<dim3((uint32_t)rows), 256, 0, st>>>(c, a, p.cut);
}

// A pool without pages hides every token.
KvAttention without_keys(const KvCache& c, const KvAttention& a) {
  KvAttention b = a;
  if (c.num_pages == 0) b.max_kv_len = b.prefix_len = 0;
  return b;
}

}  // namespace

bool kv_attention_supported(const KvCache& c, const KvAttention& a) {
  const Plan p = make_plan(c, without_keys(c, a));
  const int64_t all = (int64_t)a.batch * c.heads * p.cut.own_tiles * std::max<int64_t>(1, ceil_div(a.max_kv_len, kPass));
  // a grid holds fewer than 2^32 threads
  auto fits = [](int64_t groups, int threads) { return groups * threads <= (int64_t)UINT32_MAX; };
  const int tile_threads = c.head_dim == 64    ? Tile<64>::kThreads
                           : c.head_dim == 128 ? Tile<128>::kThreads
                                               : Tile<256>::kThreads;
  auto threads = [&](int mt) { return mt > 0 ? 256 : tile_threads; };
  const bool one_launch = p.prefix_items == 0 || p.prefix_mt == p.own_mt;
  return all <= (INT32_MAX >> 1) && fits(p.own_items + (one_launch ? p.prefix_items : 0), threads(p.own_mt)) &&
         fits(p.prefix_items, threads(p.prefix_mt)) && (p.parts == 0 || fits(ceil_div(a.total_q * a.q_heads, 4), 256));
}

int64_t kv_attention_workspace_bytes(const KvCache& c, const KvAttention& a) {
  if (a.total_q <= 0) return 0;
  return make_plan(c, without_keys(c, a)).parts * (8 + 4 * (int64_t)c.head_dim);
}

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, void* workspace, hipStream_t stream) {
  const KvAttention b = without_keys(c, a);
  Plan p = make_plan(c, b);
  // the values first: they keep 16-byte alignment
  p.cut.part_o = (float*)workspace;
  p.cut.part_ml = p.cut.part_o + p.parts * c.head_dim;
  if (c.head_dim == 64) run_attention<64>(c, b, p, stream);
  else if (c.head_dim == 128) run_attention<128>(c, b, p, stream);
  else run_attention<256>(c, b, p, stream);
  return hipGetLastError();
}

}  // namespace nvfp4k
