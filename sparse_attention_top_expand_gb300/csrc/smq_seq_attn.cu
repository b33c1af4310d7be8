// Attention of sequences' query rows over a paged key-value cache (sm_103a): a
// sliding window with sinks, or a tree of drafted tokens.
//
// An item is a block of a sequence's rows on one kv head. Its rows and their
// query heads are the M side of the products: a tile of 128 holds 128 / G rows
// with G heads each. Over tiles of 128 tokens,
//   S = Q K^T       tcgen05.mma, M = 128 queries, N = 128 tokens, to TMEM
//   P = 2^(c S - m) a thread owns one query: no value crosses threads
//   O += P V        tcgen05.mma with P read from TMEM, where it replaces S
// with a running maximum m and sum l per thread, in one pass over the tokens.
// m is raised only when a score exceeds it by kTau (in log2), so the rescale of
// O stays out of the common path.
//
// Two streams, each with its own S, P and O in TMEM, its own softmax group and
// its own product warp, keep the tensor core busy: one stream's products run
// behind the other's softmax. Where sequences have more queries than a tile
// (kPair) the streams are two tiles of queries, and each key and value is read
// once for both. Otherwise they are one tile of queries over every other tile of
// tokens, joined in TMEM.
//
// Rounding. Queries, keys and values go to the tensor core as they are held: bf16,
// and E4M3 codes widened to bf16, which is exact. S, m, l and O are fp32. P is
// rounded to bf16 (times its token's value scale before that): 2^-8 of a weight at
// most, some 0.0015 of a result's norm beside the 0.0017 of its own rounding. Two
// numbers a weight, as in smq_attn.cu, would be half as many products again, and
// these are what a prefill's time is made of. Calls of few rows have time for them,
// but the tensor core cuts what a step adds at 2^-24 of the sum so far, and twice
// the steps with parts of 2^-8 lose more to that than a long context can spare:
// 2^31 equal scores gave 0.93 for 1, with one number a weight 1.
//
// What a row does not see. Scores of tokens that are not there, or not seen, are
// minus infinity, so their weights are zeros. That does not keep out an infinite
// value, or NaN, of a token that other rows of the tile see. So a warp looks
// through the values of the tokens that some row of its own does not see, of a
// masked tile only; where one is not finite it sums that tile for its rows by
// hand, with each row's own tokens, in place of the product. The work is that of
// the tile (some 160 us), whatever the context's length.
//
// Split. The tiles of all items form one list, cut into equal ranges, one per CTA
// and SM, whatever the lengths are. A range that starts or ends inside an item
// leaves an unnormalised partial in the workspace, and seq_combine_kernel joins
// those of an item in the order of the list: results do not depend on timing.
//
// Roles: warps 0-3 copy K, V and Q (cp.async; over an E4M3 cache they bring keys
// and warps 16-19 values, and widen them), warp 4 cuts the work into segments,
// warps 5 and 7 issue the products, warp 6 looks up addresses, warps 8-15 are the
// softmax.
//
// What bounds it. A pair of tiles (256 queries by 128 tokens, D 128) is 2048 cycles
// of products at the tensor core's rate and takes some 3500: S to P, P to the next
// S and the hand-offs between are a chain that two streams do not cover. The
// roles run from one instruction cache, and the size of the softmax's loop decides,
// of code in it that is read past too. 4096 rows, 64 heads on 8, a window of 4096
// take 468 to 476 us, 1.16 to 1.17 PFLOP/s, 60 % of what a library's product of
// 8192^3 reaches; on kernels of their days 536 with the 128 scores of a thread in
// registers, and against 454 in loops of 32 tokens that read S from TMEM twice 532
// in loops of 64, 516 in loops of 16, and 552 to 607 with the next 32 asked for ahead.
//  - trees of 64 tokens over contexts of 4096 to 32768, 16 sequences, the same
//    heads: 504 to 543 us, 1.13 to 1.22 PFLOP/s.
//  - 64 sequences of up to 4 rows, a window of 4096, E4M3: 251 us for 567 MB; a
//    tile of 128 tokens takes 3300 cycles, of which a loader warp 1400 to widen
//    its part and 1100 to copy the next (twice as many loader warps: the same), and
//    every product has 128 queries' rows, of which 8 to 32 are there.
//  - small calls, 16 to 19 us: three dependent loads to the first key (sequence,
//    block table, cache), one tile's chain, the join (a launch of its own).
#include "smq_attn.cuh"
#include "smq_attn_ptx.cuh"
#include "smq_kernels.cuh"
#include "smq_ptx.cuh"

#include <type_traits>

namespace smq {

namespace {

constexpr int kLoaders = 128;  // threads that copy K, V and Q; over an E4M3 cache these keys and queries, as many again values
constexpr int kSegRing = 8;    // segments published ahead
constexpr int kRing = 4;       // tiles whose addresses, masks and scales may be ahead of the softmax
constexpr float kUnset = -3.402823466e38f;  // the running maximum of a partial without tokens: no score is below it
constexpr float kFar = 134217728.f;        // 2^27: a maximum whose rounding a fused scale and maximum would show as a factor of 2^4
constexpr int kSmemLimit = 232448 - 1024;  // less the static part
constexpr float kTau = 8.f;                // log2 of the largest P

// A run of token tiles of one item. The item's tokens are numbered e = 0 .. count - 1: position e below s0, e + gap from
// there on.
struct SeqSeg {
  int32_t row0, nrows;    // rows of q and out
  int32_t kvh;
  int32_t tile0, ntiles;  // ntiles = 0: the end of this CTA's work
  int32_t slot;           // partial slot, -1: the whole item, write the result
  int32_t table_row;      // of the block table, -1: out of range
  int32_t s0, gap, count;
  int32_t end0;           // window: position of the first row, plus one; tree: tokens before the drafted ones
  int32_t pad[5];
};
static_assert(sizeof(SeqSeg) == 64, "");

// A kernel's shapes. Shared memory holds the queries, kSlots tiles of K or V as the tensor core reads them, over an E4M3
// cache kRaws tiles of codes of each side, and the rings.
template <int D, bool kE4m3, bool kPair>
struct SeqShape {
  static constexpr int kBlocks = D / 64;                 // 128-byte columns of a token
  static constexpr int kUnit = kBlocks * 128 * 128;      // bytes of a K, V or Q tile
  static constexpr int kRaw = kE4m3 ? 128 * D : 0;       // bytes of a tile's codes
  static constexpr int kQBytes = (kPair ? 2 : 1) * kUnit;
  static constexpr int kQueries = kPair ? kSeqQueries : 128;
  static constexpr int kThreads = kE4m3 ? 640 : 512;
  // registers of a thread: at launch all of an SM's, then most for the 256 softmax threads
  static constexpr int kRegs = kE4m3 ? 96 : 128;
  static constexpr int kSoftmaxRegs = kE4m3 ? 152 : 184;
  static constexpr int kOtherRegs = kE4m3 ? 56 : 72;
  static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kRegs, "");
  static constexpr int kStep = 32;  // tokens that a softmax thread takes at a time
  static constexpr int kAddrReaders = (kE4m3 ? 8 : 4) + (kPair ? 8 : 4);  // loader and softmax warps of a tile
  static constexpr int kSegReaders = (kE4m3 ? 8 : 4) + 8 + 3;             // and MMA and address warps
  static constexpr int kRingBytes = kRing * 128 * (8 + (kE4m3 ? 8 : 0)) + kRing * 16;
  static constexpr int kBarBytes = 576;
  static constexpr int kMisc = kRingBytes + kSegRing * 64 + kBarBytes + 2 * 128 * 8 /*m and l*/;
  static constexpr int kFree = kSmemLimit - kQBytes - kMisc;
  // over an E4M3 cache one or two units of each side (each side's loaders keep to slots of their own, so that a wait's
  // parity names one phase), so that what is left over goes to the copies ahead
  static constexpr int kFit = kE4m3 ? (kFree >= 4 * kUnit + 4 * kRaw ? 4 : 2) : kFree / kUnit;
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;
  static constexpr int kRawFit = kE4m3 ? (kFree - kSlots * kUnit) / (kE4m3 ? 2 * kRaw : 1) : 0;
  static constexpr int kRaws = kRawFit > 4 ? 4 : kRawFit;  // of each side
  static constexpr int kSmem = kSlots * kUnit + 2 * kRaws * kRaw + kQBytes + kMisc;
  static constexpr int kTmem = 512;                        // two S (P takes its place), two O
  static_assert((kE4m3 ? kSlots % 2 == 0 && kRaws >= 1 : kSlots >= 3) && kSlots <= 8 && kSmem <= kSmemLimit, "");
};

// Instruction descriptor of O += P V: fp32 accumulation, bf16 operands, N-major B, M = 128.
__host__ __device__ constexpr uint32_t pv_idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

// D[tmem] (+)= A[tmem] x B; b is a descriptor's two words.
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n mov.b64 y, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* x) {
  uint32_t v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(x[i]);
  tmem_st16(taddr, v);
  tmem_st16(taddr + 16, v + 16);
}

// Sequence b: its first row, rows and length; no rows where it is refused.
struct Sequence {
  int32_t first, rows, len;
};
__device__ __forceinline__ Sequence sequence_of(const SeqAttnParams& p, int b, bool report) {
  Sequence s;
  const int32_t last = p.cu_rows[b + 1];
  s.first = p.cu_rows[b];
  s.rows = 0;
  s.len = max(p.seq_len[b], 0);
  if (s.first < 0 || last < s.first || last > p.rows || last - s.first > p.max_seq_rows) {
    if (report) atomicOr(p.status, kStatusBounds);
  } else {
    s.rows = last - s.first;
  }
  return s;
}

// The tokens of rows i0 .. i0 + rows - 1 of a sequence: positions [0, s0) and [lo, hi).
struct Tokens {
  int32_t s0, lo, hi;
  bool past;  // the rows' last token (of a tree: the sequence's) is past the block table
  __device__ int32_t count() const { return s0 + hi - lo; }
  // (without tokens there still is a result; up to 2^31 - 1 tokens, so nothing is added to a count or a token's number)
  __device__ int32_t tiles() const { return (count() - 1) / kAttnTile + 1; }
};
__device__ __forceinline__ Tokens tokens_of(const SeqAttnParams& p, int32_t n, int32_t len, int32_t i0, int32_t rows) {
  const int64_t room = static_cast<int64_t>(p.bt_stride) * p.page_size;
  const int32_t cap = room > INT32_MAX ? INT32_MAX : static_cast<int32_t>(room);
  Tokens t;
  const int32_t last = p.tree_mask ? len : len - n + i0 + rows;
  t.hi = min(max(last, 0), cap);
  t.past = last > cap;
  t.lo = 0;
  if (!p.tree_mask) {
    const int32_t first = len - n + i0 + 1;
    t.lo = min(first > p.window ? first - p.window : 0, t.hi);
  }
  t.s0 = min(p.sinks, t.lo);
  return t;
}

// Whether rows i0 .. i0 + rows - 1 of a sequence see a token past the block table's `cap` positions, given that its last one
// is: of a tree its context, or a drafted token whose bit one of them has. A warp's call, a lane's answer. (Inlined it costs
// a prefill 5 % of its time, though it is not run: the roles share one instruction cache.)
__device__ __noinline__ bool sees_past(const SeqAttnParams& p, Sequence s, int32_t i0, int32_t rows, int32_t cap, int lane) {
  const int32_t base = s.len - s.rows;
  if (!p.tree_mask || base > cap) return true;
  const int32_t node = cap - base;  // the first one past the table
  bool sees = false;
  for (int r = lane; r < rows; r += 32) {
    const int32_t* const words = p.tree_mask + (static_cast<int64_t>(s.first) + i0 + r) * p.mask_words;
    for (int i = node >> 5; i < p.mask_words && i * 32 < s.rows; ++i) {
      uint32_t bits = words[i];
      if (i == node >> 5) bits &= 0xffffffffu << (node & 31);
      if (s.rows - i * 32 < 32) bits &= (1u << (s.rows - i * 32)) - 1u;
      sees |= bits != 0;
    }
  }
  return sees;
}

// What row r of an item sees of a window, in the item's numbering: [0, x) and [y, z).
__device__ __forceinline__ void row_sees(const SeqAttnParams& p, const SeqSeg& sg, int r, int32_t& x, int32_t& y, int32_t& z) {
  const int32_t end = sg.end0 + r;
  z = end - sg.gap;
  y = (end > p.window ? end - p.window : 0) - sg.gap;
  x = sg.gap > 0 ? sg.s0 : min(p.sinks, z);
}

// Bits of the tokens below x among the 32 from e on.
__device__ __forceinline__ uint32_t bits_below(int32_t x, int32_t e) {
  return x <= e ? 0u : x - e >= 32 ? 0xffffffffu : (1u << (x - e)) - 1u;
}

// Which of the 32 tokens from e on row r of an item sees (of those that are there).
__device__ __forceinline__ uint32_t seen_by(const SeqAttnParams& p, const SeqSeg& sg, int32_t e, int r) {
  if (!p.tree_mask) {
    int32_t x, y, z;
    row_sees(p, sg, r, x, y, z);
    return bits_below(x, e) | (bits_below(z, e) & ~bits_below(y, e));
  }
  uint32_t v = bits_below(sg.end0, e);
  const int32_t node = e - sg.end0;  // of the first token
  if (node > -32 && r < sg.nrows) {
    const int32_t* const words = p.tree_mask + (static_cast<int64_t>(sg.row0) + r) * p.mask_words;
    const int i = node >> 5;  // (rounds down)
    const uint32_t lo = i >= 0 && i < p.mask_words ? words[i] : 0;
    const uint32_t hi = i + 1 < p.mask_words ? words[i + 1] : 0;
    v |= __funnelshift_r(lo, hi, node & 31);
  }
  return v;
}

// Whether a value is not finite among those of `tokens` (bits) of the 32 from t0 on of a unit of values; a warp's call, each
// lane's answer is of its pieces.
template <int D>
__device__ __forceinline__ bool not_finite(uint32_t unit, uint32_t tokens, int t0, int lane) {
  constexpr int kChunks = D / 8, kTok = 32 / kChunks;  // 16-byte pieces of a token, tokens per warp instruction
  const int piece = lane % kChunks, sub = lane / kChunks;
  const uint32_t base = unit + (piece >> 3) * 16384 + (t0 + sub) * 128;
  __nv_bfloat162 most = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < 32; i += kTok) {
    uint32_t w[4];
    lds16(base + i * 128 + (((piece & 7) ^ ((i + sub) & 7)) << 4), w);
    const uint32_t keep = (tokens >> (i + sub)) & 1 ? 0x7fff7fffu : 0u;  // without signs
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] &= keep;
      most = __hmax2_nan(most, *reinterpret_cast<const __nv_bfloat162*>(w + k));
    }
  }
  const uint32_t m = *reinterpret_cast<const uint32_t*>(&most);
  return (m & 0x7f80u) == 0x7f80u || (m & 0x7f800000u) == 0x7f800000u;
}

// A masked tile by hand, in fp32, for a warp's rows: O so far (zero for the `first` tile) and the values of the tokens that
// each row sees. The product of the tile, which the other warps' rows need, goes ahead, and what it makes of these rows is
// replaced. False where a wait ran out. bars: P written, addresses free, and the product done, of this tile and, with the
// other parity, of the one before.
template <int D>
__device__ __noinline__ bool tile_by_hand(uint32_t p_col, uint32_t o_col, uint32_t unit, const uint32_t* seen, bool first,
                                          uint32_t p_full, uint32_t a_empty, uint32_t pv_done, uint32_t parity,
                                          const volatile int* abort, uint64_t limit) {
  const int lane = threadIdx.x & 31;
  if (!first && !wait_phase(pv_done, parity ^ 1, abort, limit)) return false;
  tc_fence_after();
  float w[64], sum[D];  // (local memory)
#pragma unroll 1
  for (int c = 0; c < 64; c += 16) {
    float x[16];
    tmem_ld<16>(p_col + c, x);
    tmem_wait_ld();
    pin<16>(x);
    for (int i = 0; i < 16; ++i) w[c + i] = x[i];
  }
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    float o[16];
    tmem_ld<16>(o_col + c, o);
    tmem_wait_ld();
    pin<16>(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = first ? 0.f : o[i];
#pragma unroll 1
    for (int t = 0; t < 128; ++t) {
      uint32_t v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        lds16(unit + (c >> 6) * 16384 + t * 128 + (((((c & 63) >> 3) + h) ^ (t & 7)) << 4), v + 4 * h);
      if (!((seen[t >> 5] >> (t & 31)) & 1)) continue;
      const uint32_t pair = __float_as_uint(w[t >> 1]);
      const float p = __uint_as_float(t & 1 ? pair & 0xffff0000u : pair << 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[2 * i] = fmaf(p, __uint_as_float(v[i] << 16), o[2 * i]);
        o[2 * i + 1] = fmaf(p, __uint_as_float(v[i] & 0xffff0000u), o[2 * i + 1]);
      }
    }
    __syncwarp();
    for (int i = 0; i < 16; ++i) sum[c + i] = o[i];
  }
  tc_fence_before();
  __syncwarp();
  arrive_one(p_full, lane);
  arrive_one(a_empty, lane);
  if (!wait_phase(pv_done, parity, abort, limit)) return false;
  tc_fence_after();
#pragma unroll 1
  for (int c = 0; c < D; c += 8) {
    float x[8];
    for (int i = 0; i < 8; ++i) x[i] = sum[c + i];
    tmem_st8(o_col + c, x);
  }
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  return true;
}

// A tile's weights where a maximum is past kFar: score times scale is rounded before the maximum is taken off, as the maximum
// was, since a fused one would show the maximum's rounding as a factor. By each query's own maximum, so that equal scores weigh
// alike in all tiles. The sum of this thread's weights.
template <bool kE4m3>
__device__ __noinline__ float far_weights(uint32_t s_col, const float* k_scales, const float* v_scales, bool scaled, float scale,
                                          float nm) {
  const bool apart = fabsf(nm) > kFar;
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < 128; c += 16) {
    float x[16];
    tmem_ld<16>(s_col + c, x);
    tmem_wait_ld();
    pin<16>(x);
    float w[8];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (kE4m3 && !scaled) x[i] *= k_scales[c + i];
      x[i] = ex2(apart ? __fadd_rn(__fmul_rn(x[i], scale), nm) : fmaf(x[i], scale, nm));
      sum += x[i];
      if (kE4m3) x[i] *= v_scales[c + i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __uint_as_float(bf16x2(x[2 * i], x[2 * i + 1]));
    tmem_st8(s_col + c / 2, w);
  }
  tmem_wait_st();
  return sum;
}

}  // namespace

template <int D, bool kE4m3, bool kPair>
__global__ void __launch_bounds__(SeqShape<D, kE4m3, kPair>::kThreads, 1)
    seq_attention_kernel(const __grid_constant__ SeqAttnParams p) {
  using S = SeqShape<D, kE4m3, kPair>;
  constexpr int kThreads = S::kThreads;
  extern __shared__ __align__(1024) uint8_t smem[];
  // operands first (1024-byte aligned), then rings, state and barriers
  uint8_t* const units = smem;
  uint8_t* const q_s = units + S::kSlots * S::kUnit;
  uint8_t* const raws = q_s + S::kQBytes;                                              // E4M3
  int64_t* const ring_off = reinterpret_cast<int64_t*>(raws + 2 * S::kRaws * S::kRaw);  // [ring][128]
  float* const ring_ks = reinterpret_cast<float*>(ring_off + kRing * 128);             // [ring][128], E4M3
  float* const ring_vs = ring_ks + (kE4m3 ? kRing * 128 : 0);
  uint32_t* const ring_mask = reinterpret_cast<uint32_t*>(ring_vs + (kE4m3 ? kRing * 128 : 0));  // [ring][4]
  SeqSeg* const segs = reinterpret_cast<SeqSeg*>(ring_mask + kRing * 4);
  float2* const ml_s = reinterpret_cast<float2*>(segs + kSegRing);  // [2][128] maxima and sums to be joined
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ml_s + 256);
  // kFull: keys, then values, of a stream's tile n (with kPair of both streams'): four each, as many as there may be tiles ahead,
  // all of which can be one stream's, so that a wait's parity names one phase
  constexpr int kFull = 0, kEmpty = kFull + (kPair ? 8 : 16), kSFull = kEmpty + S::kSlots, kPFull = kSFull + 2, kPvDone = kPFull + 2,
                kJoin = kPvDone + 2, kQEmpty = kJoin + 1, kQFull = kQEmpty + 1, kSegFull = kQFull + 1,
                kSegEmpty = kSegFull + kSegRing, kAFull = kSegEmpty + kSegRing, kAEmpty = kAFull + kRing,
                kDrain = kAEmpty + kRing, kScFull = kDrain + 2, kBars = kScFull + (kE4m3 ? kRing : 0);
  static_assert(kBars * 8 <= S::kBarBytes && kBars <= kThreads, "");
  auto bar = [&](int i) { return smem_addr(bars + i); };
  static_assert(S::kSlots <= 8, "");
  auto full_bar = [](int stream, int side, uint32_t n) {
    return kFull + ((kPair ? 0 : stream) * 2 + side) * 4 + static_cast<int>(n & 3);
  };
  auto full_parity = [](uint32_t n) { return (n >> 2) & 1; };

  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ long long warp_sum[kThreads / 32];
  __shared__ int start_seq;
  __shared__ long long start_idx;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t limit = static_cast<uint64_t>(p.wait_ns);
  griddep_launch_dependents();

  if (tid < kBars) {  // a barrier a thread
    const int i = tid;
    const int count = i < kEmpty ? (kE4m3 ? kLoaders / 32 : kLoaders)   // K and V units: loader warps, or each thread's copies
                      : i < kSFull ? (kPair ? 2 : 1)                    // freed by the MMAs of each stream that reads them
                      : i < kPFull ? 1                                  // S
                      : i < kPvDone ? 4                                 // P written: each softmax warp
                      : i < kJoin ? 1 : i < kQEmpty ? 8                 // O; both streams' results
                      : i < kQFull ? 2 : i < kSegFull ? kLoaders        // queries: freed by both streams; E4M3: each thread's copies
                      : i < kSegEmpty ? 1 : i < kAFull ? S::kSegReaders // segments
                      : i < kAEmpty ? 1 : i < kDrain ? S::kAddrReaders  // addresses
                      : i < kScFull ? 1 : 64;                           // drains; scales: each lane's copies, and its stores
    mbar_init(bar(i), count);
    mbar_init_fence();
  }
  if (tid == 0) {
    abort_flag = 0;
    start_seq = -1;
  }
  if (warp == 5) tmem_alloc(smem_addr(&tmem_slot), S::kTmem);
  griddep_wait();

  // ---- this CTA's range of the tile list: sequences, kv heads, blocks of rows, tiles
  tc_fence_before();
  const int per_tile = 128 / p.group, per_item = (kPair ? 2 : 1) * per_tile;  // rows of a tile of queries, and of an item
  // tiles of this lane's sequence on one kv head
  auto tiles_of = [&](const Sequence& s) {
    long long mine = 0;
    if (s.rows > 0 && s.rows <= per_item) mine = tokens_of(p, s.rows, s.len, 0, s.rows).tiles();
    for (uint32_t many = __ballot_sync(0xffffffffu, s.rows > per_item); many; many &= many - 1) {
      const int src = __ffs(many) - 1;
      const int n = __shfl_sync(0xffffffffu, s.rows, src), len = __shfl_sync(0xffffffffu, s.len, src);
      long long wide = 0;
      for (int i = lane * per_item; i < n; i += 32 * per_item) wide += tokens_of(p, n, len, i, min(per_item, n - i)).tiles();
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xffffffffu, wide, o);
      if (lane == src) mine = wide;
    }
    return mine;
  };
  auto head_tiles = [&](int base, int end, bool report) {  // of sequence base + lane, for the sequences below end
    Sequence s = {0, 0, 0};
    if (base + lane < end) s = sequence_of(p, base + lane, report);
    return tiles_of(s);
  };
  auto scan_lanes = [&](long long v) {  // inclusive prefix sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    return v;
  };
  long long total = 0, chunk = 0, work = 0;  // the scheduler's, which works them out alone where a lane a sequence is enough
  if (p.num_seqs > 32) {
    constexpr int kWarps = kThreads / 32;
    const int groups = (p.num_seqs + 31) / 32, per_warp = (groups + kWarps - 1) / kWarps;
    const int seq0 = warp * per_warp * 32, seq1 = min(p.num_seqs, (warp + 1) * per_warp * 32);
    long long mine = 0;
    for (int base = seq0; base < seq1; base += 32) mine += head_tiles(base, seq1, blockIdx.x == 0);
    mine = scan_lanes(mine * p.kv_heads);
    if (lane == 31) warp_sum[warp] = mine;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    chunk = div_of(total + gridDim.x - 1, gridDim.x);
    const long long begin = chunk * blockIdx.x;
    work = begin < total ? min(chunk, total - begin) : 0;
    if (work > 0 && begin >= before && begin < before + warp_sum[warp]) {
      long long at = before;
      for (int base = seq0; base < seq1; base += 32) {
        const long long t = head_tiles(base, seq1, false) * p.kv_heads, incl = scan_lanes(t);
        if (begin >= at + incl - t && begin < at + incl) {
          start_seq = base + lane;
          start_idx = begin - (at + incl - t);
        }
        at += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const volatile int* const abort = &abort_flag;
  auto fail = [&] { *reinterpret_cast<volatile int*>(&abort_flag) = 1; };  // reported at the end

  // the softmax threads take registers that the others do not need
  if (warp < 8 || warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kOtherRegs));
    bool ok = true;
    auto wait = [&](int b, uint32_t parity) {
      ok = wait_phase(bar(b), parity, abort, limit);
      return ok;
    };
    if (warp < 4 || warp >= 16) {
      // ------------------------------------------------------------ loaders
      const int stall_tile = blockIdx.x == 0 ? p.stall_tile : -1;  // tests: its keys are not handed over
      const uint32_t units_a = smem_addr(units);
      auto fetch_queries = [&](const SeqSeg& sg) {
        constexpr int kChunks = D / 8, kQTok = 32 / kChunks;  // 16-byte pieces of a query, queries per warp instruction
        const int c = lane % kChunks;
        const uint16_t* const base = p.q + sg.row0 * p.q_stride + static_cast<int64_t>(sg.kvh) * p.group * D + c * 8;
        const uint32_t dst = smem_addr(q_s) + (c >> 3) * 16384;
        const int nrows = sg.nrows;
        const uint32_t inv = 65536 / p.group + 1;  // m * inv >> 16 is m / group for m below 128
#pragma unroll 4
        for (int i = warp * kQTok + lane / kChunks; i < S::kQueries; i += 4 * kQTok) {
          const int t = kPair ? i >> 7 : 0, m = i & 127, r = static_cast<int>(m * inv >> 16), row = t * per_tile + r;
          const bool there = r < per_tile && row < nrows;
          cp16(dst + t * S::kUnit + m * 128 + (((c & 7) ^ (m & 7)) << 4),
               base + (there ? row * p.q_stride + (m - r * p.group) * D : 0), there ? 16 : 0);
        }
        cp_arrive(bar(kQFull));
      };
      if constexpr (kE4m3) {
        // Warps 0-3 bring keys, warps 16-19 values. Each lane copies pieces of 16 codes into a place of its own and widens
        // them later into the unit that the tensor core reads, so the copies need no barrier. Two cursors go over the
        // tiles: one copies, up to kRaws tiles ahead of the one that widens.
        constexpr int kPieces = D / 16;                       // of a token
        constexpr int kTok = 32 / kPieces, kPer = 32 / kTok;  // tokens per warp instruction, pieces per lane and unit
        // Eight lanes have two neighbouring tokens' pieces of one 128-byte column, so that their stores, two 16-byte
        // chunks apart within a token and swizzled by the token, meet every bank once.
        const int piece = (lane & 3) | (kPieces == 8 ? (lane >> 1) & 4 : 0);
        const int sub = kPieces == 8 ? ((lane >> 2) & 1) | ((lane >> 3) & 2) : lane >> 2;
        const bool values = warp >= 16;
        const int w0 = (warp & 3) * 32;                       // the warp's first token
        uint8_t* const mine_raw = raws + (values ? S::kRaws * S::kRaw : 0) + w0 * D + lane * 16;
        const uint8_t* const base = static_cast<const uint8_t*>(values ? p.v_cache : p.k_cache) + piece * 16;
        int ahead = 0;                                        // tiles copied and not yet widened
        int cseg = 0, cleft = 0, ctile = 0, craw = 0;         // copying
        int seg = 0, left = 0, tile = 0, raw = 0;             // widening
        int slot = values ? 1 : 0;                            // keys in the even units, values in the odd ones
        uint32_t mine_n = 0, other_n = 0;                     // tiles so far of the next tile's stream, and of the other
        int stream = 0;
        auto swap_streams = [&] {
          stream ^= 1;
          const uint32_t x = mine_n;
          mine_n = other_n;
          other_n = x;
        };
        uint32_t turn = 1;
        bool more = true;
        auto ready = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test_wait(bar(b), parity)); };
        while (true) {
          if (more && ahead < S::kRaws) {
            // copy the next tile; as long as there is something to widen, only if its segment and addresses are there
            bool there = true;
            if (cleft == 0) {
              const int at = kSegFull + cseg % kSegRing, parity = (cseg / kSegRing) & 1;
              there = ahead > 0 ? ready(at, parity) : wait(at, parity);
              if (there) {
                cleft = segs[cseg % kSegRing].ntiles;
                more = there = cleft > 0;
                ++cseg;
              }
            }
            if (there) {
              const int at = kAFull + ctile % kRing, parity = (ctile / kRing) & 1;
              there = ahead > 0 ? ready(at, parity) : wait(at, parity);
            }
            if (!ok) break;
            if (there) {
              const int64_t* const offs = ring_off + ctile % kRing * 128 + w0 + sub;
              const uint32_t dst = smem_addr(mine_raw) + craw * S::kRaw;
              const bool whole = ring_mask[ctile % kRing * 4 + (warp & 3)] == 0xffffffffu;  // every token is there
              if (__builtin_expect(whole, 1)) {
#pragma unroll
                for (int i0 = 0; i0 < kPer; i0 += 4) {
                  const uint8_t* src[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i) src[i] = base + offs[(i0 + i) * kTok];
#pragma unroll
                  for (int i = 0; i < 4; ++i) cp16(dst + (i0 + i) * 512, src[i]);
                }
              } else {
#pragma unroll 1
                for (int i = 0; i < kPer; ++i) {
                  const int64_t o = offs[i * kTok];
                  cp16(dst + i * 512, base + (o < 0 ? 0 : o), o < 0 ? 0 : 16);
                }
              }
              cp_commit();
              __syncwarp();
              arrive_one(bar(kAEmpty + ctile % kRing), lane);
              ++ctile;
              --cleft;
              if (++craw == S::kRaws) craw = 0;
              ++ahead;
              continue;
            }
          }
          if (ahead == 0) break;
          if (left == 0) {
            left = segs[seg % kSegRing].ntiles;
            if (stream == 1) swap_streams();  // a segment begins with stream 0
            if (!values) {
              if (!wait(kQEmpty, (seg + 1) & 1)) break;
              fetch_queries(segs[seg % kSegRing]);
            }
            __syncwarp();
            arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
            ++seg;
          }
          if (!wait(kEmpty + slot, turn)) break;
          if (ahead == S::kRaws)
            cp_wait<S::kRaws - 1>();  // the oldest tile has landed
          else
            cp_wait_all();
          const uint8_t* const src = mine_raw + raw * S::kRaw;
          const uint32_t dst = units_a + slot * S::kUnit + (piece >> 2) * 16384 + (w0 + sub) * 128;
#pragma unroll 1
          for (int i0 = 0; i0 < kPer; i0 += 2) {
            uint4 w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) w[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * 512);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t row = dst + (i0 + i) * (kTok * 128), t = (i * kTok + sub) & 7;  // i0 * kTok is a multiple of 8
              uint32_t x[4];
              widen4(w[i].x, x[0], x[1]);
              widen4(w[i].y, x[2], x[3]);
              sts16(row + (((piece & 3) * 2 ^ t) << 4), x[0], x[1], x[2], x[3]);
              widen4(w[i].z, x[0], x[1]);
              widen4(w[i].w, x[2], x[3]);
              sts16(row + (((piece & 3) * 2 + 1 ^ t) << 4), x[0], x[1], x[2], x[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (values || stall_tile != tile) arrive_one(bar(full_bar(stream, values, mine_n)), lane);
          ++mine_n;
          if (!kPair) swap_streams();
          slot += 2;
          if (slot >= S::kSlots) {
            slot -= S::kSlots;
            turn ^= 1;
          }
          if (++raw == S::kRaws) raw = 0;
          --ahead;
          ++tile;
          --left;
        }
      } else {
        constexpr int kChunks = D / 8;      // 16-byte pieces of a token
        constexpr int kTok = 32 / kChunks;  // tokens per warp instruction
        const int piece = lane % kChunks, sub = lane / kChunks;
        // Units: K 0, V 0, K 1, V 1, ... The unit's barrier counts each thread's copies when they land; the MMA warp's
        // proxy fence, after its wait, orders them before the tensor core's reads.
        int slot = 0, seg = 0, left = 0, tile = 0;  // left: tiles of this segment
        bool asked = true;                          // its queries are on their way
        uint32_t turn = 1;                          // parity that says that the slot is free
        uint32_t mine_n = 0, other_n = 0;           // tiles so far of the next tile's stream, and of the other
        int stream = 0;
        auto swap_streams = [&] {
          stream ^= 1;
          const uint32_t x = mine_n;
          mine_n = other_n;
          other_n = x;
        };
        auto ask = [&](int& at, bool& done) {
          fetch_queries(segs[at % kSegRing]);
          __syncwarp();
          arrive_one(bar(kSegEmpty + at % kSegRing), lane);
          ++at;
          done = true;
        };
        for (bool values = false; ok; values = !values) {
          if (!values) {
            if (left == 0) {
              if (stream == 1) swap_streams();  // a segment begins with stream 0
              if (!wait(kSegFull + seg % kSegRing, (seg / kSegRing) & 1)) break;
              left = segs[seg % kSegRing].ntiles;
              if (left == 0) break;
              asked = false;
            }
            if (!wait(kAFull + tile % kRing, (tile / kRing) & 1)) break;
          }
          // the segment's queries, as soon as their place is free; its first tile need not wait for that
          if (!asked && __all_sync(0xffffffffu, mbar_test_wait(bar(kQEmpty), (seg + 1) & 1))) ask(seg, asked);
          if (!wait(kEmpty + slot, turn)) break;
          const uint8_t* const base = static_cast<const uint8_t*>(values ? p.v_cache : p.k_cache) + piece * 16;
          const int64_t* const offs = ring_off + tile % kRing * 128 + warp * 32 + sub;
          constexpr int kBatch = 32 / kTok < 8 ? 32 / kTok : 8;  // addresses first, so that the copies issue back to back
          const uint32_t dst = units_a + slot * S::kUnit + (piece >> 3) * 16384 + (warp * 32 + sub) * 128;
          const bool whole = ring_mask[tile % kRing * 4 + warp] == 0xffffffffu;  // every token of the warp is there
          if (__builtin_expect(whole, 1)) {
#pragma unroll
            for (int i0 = 0; i0 < 32 / kTok; i0 += kBatch) {
              const uint8_t* src[kBatch];
#pragma unroll
              for (int i = 0; i < kBatch; ++i) src[i] = base + offs[(i0 + i) * kTok];
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
                cp16(dst + (i0 + i) * kTok * 128 + (((piece & 7) ^ (((i0 + i) * kTok + sub) & 7)) << 4), src[i]);
            }
          } else {
#pragma unroll 1
            for (int i0 = 0; i0 < 32 / kTok; i0 += 4) {
              int64_t o[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = offs[(i0 + i) * kTok];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                cp16(dst + (i0 + i) * kTok * 128 + (((piece & 7) ^ (((i0 + i) * kTok + sub) & 7)) << 4),
                     base + (o[i] < 0 ? 0 : o[i]), o[i] < 0 ? 0 : 16);
            }
          }
          if (values || stall_tile != tile) cp_arrive(bar(full_bar(stream, values, mine_n)));
          if (++slot == S::kSlots) {
            slot = 0;
            turn ^= 1;
          }
          if (values && !asked) {
            if (!wait(kQEmpty, (seg + 1) & 1)) break;
            ask(seg, asked);
          }
          if (values) {
            __syncwarp();
            arrive_one(bar(kAEmpty + tile % kRing), lane);
            ++tile;
            --left;
            ++mine_n;
            if (!kPair) swap_streams();
          }
        }
      }
      if (!ok && lane == 0) fail();
      cp_wait_all();
    } else if (warp == 4) {
      // ---------------------------------------------------------- scheduler
      int b = 0, g = 0, k = 0, tile0 = 0;  // sequence, kv head, block, and tile of the block
      int base = -64;                      // sequences base .. base + 31 are held, one a lane
      Sequence mine_s = {0, 0, 0}, s = {0, 0, 0};
      int32_t mine_t = 0, table_row = 0;
      auto load = [&](int at) {  // sequence `at`
        if (at >= base + 32 || at < base) {
          base = at;
          mine_s = {0, 0, 0};
          if (at + lane < p.num_seqs) {
            mine_s = sequence_of(p, at + lane, p.num_seqs <= 32 && blockIdx.x == 0);
            mine_t = p.seq_indices ? p.seq_indices[at + lane] : at + lane;
            if (mine_t < 0 || mine_t >= p.bt_rows) mine_t = -1;
          }
        }
        s.first = __shfl_sync(0xffffffffu, mine_s.first, at - base);
        s.rows = __shfl_sync(0xffffffffu, mine_s.rows, at - base);
        s.len = __shfl_sync(0xffffffffu, mine_s.len, at - base);
        table_row = __shfl_sync(0xffffffffu, mine_t, at - base);
      };
      long long idx = 0, per_head = 1;  // the first segment's place within its sequence
      if (p.num_seqs <= 32) {
        load(0);
        const long long t = tiles_of(mine_s), incl = scan_lanes(t * p.kv_heads);
        total = __shfl_sync(0xffffffffu, incl, 31);
        chunk = div_of(total + gridDim.x - 1, gridDim.x);
        const long long begin = chunk * blockIdx.x;
        work = begin < total ? min(chunk, total - begin) : 0;
        const uint32_t here = __ballot_sync(0xffffffffu, begin >= incl - t * p.kv_heads && begin < incl);
        if (here) b = __ffs(here) - 1;
        idx = __shfl_sync(0xffffffffu, begin - (incl - t * p.kv_heads), b);
        per_head = __shfl_sync(0xffffffffu, t, b);
      } else if (work > 0) {
        b = start_seq;
        idx = start_idx;
        per_head = __shfl_sync(0xffffffffu, head_tiles(b, b + 1, false), 0);
      }
      long long left = work;
      if (work > 0) {
        load(b);
        g = static_cast<int>(div_of(idx, per_head));
        idx -= g * per_head;
        for (bool found = false; !found && k * per_item < s.rows; k += found ? 0 : 32) {
          const int i = (k + lane) * per_item;
          const long long t = i < s.rows ? tokens_of(p, s.rows, s.len, i, min(per_item, s.rows - i)).tiles() : 0;
          const long long incl = scan_lanes(t);
          const uint32_t here = __ballot_sync(0xffffffffu, idx >= incl - t && idx < incl);
          const int src = here ? __ffs(here) - 1 : 31;
          const long long skip = __shfl_sync(0xffffffffu, here ? incl - t : incl, src);
          idx -= skip;
          if (here) {
            k += src;
            found = true;
          }
        }
        tile0 = static_cast<int>(idx);
      }
      int4 info = make_int4(0, 0, 0, 0);
      int seg = 0;
      while (ok) {
        SeqSeg sg;
        sg.ntiles = 0;
        if (left > 0) {
          const int i0 = k * per_item, rows = min(per_item, s.rows - i0);
          const Tokens tk = tokens_of(p, s.rows, s.len, i0, rows);
          const int t = tk.tiles();
          if (tk.past && sees_past(p, s, i0, rows, tk.hi, lane)) atomicOr(p.status, kStatusBounds);
          sg.row0 = s.first + i0;
          sg.nrows = rows;
          sg.kvh = g;
          sg.tile0 = tile0;
          sg.ntiles = static_cast<int>(min(static_cast<long long>(t - tile0), left));
          sg.table_row = table_row;
          sg.s0 = tk.s0;
          sg.gap = tk.lo - tk.s0;
          sg.count = tk.count();
          sg.end0 = p.tree_mask ? s.len - s.rows : s.len - s.rows + i0 + 1;
          const bool starts = tile0 == 0, ends = tile0 + sg.ntiles == t;
          sg.slot = starts && ends ? -1 : 2 * static_cast<int>(blockIdx.x) + (starts ? 1 : 0);
          if (starts && !ends) info = make_int4(sg.row0, rows, g, static_cast<int>(div_of(t - sg.ntiles + chunk - 1, chunk)));
          left -= sg.ntiles;
          tile0 += sg.ntiles;
          if (ends) {
            tile0 = 0;
            if (++k * per_item >= s.rows) {
              k = 0;
              if (++g == p.kv_heads) {
                g = 0;
                while (left > 0) {  // (there is another sequence as long as there is work)
                  if (++b >= p.num_seqs) left = 0;
                  load(b);
                  if (s.rows > 0) break;
                }
              }
            }
          }
        }
        if (seg >= kSegRing) wait(kSegEmpty + seg % kSegRing, (seg / kSegRing - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          segs[seg % kSegRing] = sg;
          mbar_arrive(bar(kSegFull + seg % kSegRing));
        }
        __syncwarp();
        ++seg;
        if (sg.ntiles == 0) break;
      }
      if (lane == 0) {
        if (!ok) fail();
        p.seg_info[blockIdx.x] = info;
      }
    } else if (warp != 6) {
      // ---------------------------------------------------------------- MMA
      // A warp for each stream, so that neither waits for the other's softmax. The whole warp runs the loop, so that
      // descriptors stay in uniform registers, and one elected thread issues. The products of one thread with one kind and M
      // run in the order in which they are issued: S of a tile may follow the product that reads P from its place.
      constexpr uint32_t kRowHi = desc_hi(128);
      const int st = warp == 5 ? 0 : 1;
      const uint32_t units_a = smem_addr(units), q_lo = desc_lo(smem_addr(q_s) + (kPair ? st * S::kUnit : 0), 16);
      const uint32_t s_at = tmem + st * 128, o_at = tmem + 256 + st * D;
      // a negative softmax scale turns the queries round, so that the largest product is the largest score
      const uint32_t idesc = mma_idesc(false, 128) | (p.negate ? 1u << 13 : 0u);
      constexpr int step = kPair ? 1 : 2;
      uint32_t done = 0;  // tiles of this stream
      uint32_t unit = 0;  // K of the segment's first tile
      bool issued = false;
      auto slot_of = [&](uint32_t u) { return static_cast<int>(u % S::kSlots); };
      auto full = [&](int side, uint32_t n) { return wait(full_bar(st, side, n), full_parity(n)); };
      for (int seg = 0; ok; ++seg) {
        if (!wait(kSegFull + seg % kSegRing, (seg / kSegRing) & 1)) break;
        const int n = segs[seg % kSegRing].ntiles;
        // Stream 1 has nothing to do: no queries, or no tile. It gives no sign for the queries' place then, as it could be a
        // segment ahead: stream 0 gives two.
        const bool alone = kPair ? segs[seg % kSegRing].nrows <= per_tile : n == 1;
        __syncwarp();
        arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
        if (n == 0) break;
        if (alone && st == 1) {
          // as if it had read the units: each when it is there, so that its phases pass one by one
          if (kPair)
            for (uint32_t u = unit; u < unit + 2 * n && full(u & 1, u >> 1); ++u) arrive_one(bar(kEmpty + slot_of(u)), lane);
        } else {
          // O += P V of tile j, and S = Q K^T of this stream's next tile behind it
          for (int j = st * (kPair ? 0 : 1) - step; j < n; j += step) {
            const uint32_t v = unit + 2 * j + 1, k = unit + 2 * (j + step);
            const bool values = j >= 0, scores = j + step < n;
            const uint32_t nv = kPair ? v >> 1 : done;  // the tile's number at its barriers, and the next one's
            if ((values && !full(1, nv)) || (scores && !full(0, kPair ? k >> 1 : done + values))) break;
            // The queries' parity names this segment's phase only because its first keys, which were asked for behind the queries
            // of the segment before, have landed: stream 1 may have left that segment out.
            if (!values && !wait(kQFull, seg & 1)) break;
            fence_proxy_async_smem();
            if (values && !wait(kPFull + st, done & 1)) break;
            tc_fence_after();
            const uint32_t v_lo = desc_lo(units_a + slot_of(v) * S::kUnit, 16384), k_lo = desc_lo(units_a + slot_of(k) * S::kUnit, 16);
            if (elect_one()) {
              if (values) {
#pragma unroll
                for (int i = 0; i < 8; ++i)  // 16 tokens
                  mma_tmem_a(o_at, s_at + i * 8, v_lo + ((i * 16 * 128) >> 4), kRowHi, pv_idesc(D), j < step && i == 0 ? 0 : 1);
                if (!scores) mma_commit(bar(kPvDone + st));
              }
              if (scores) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  const uint32_t at = ((i >> 2) * 16384 + (i & 3) * 32) >> 4;
                  mma(s_at, q_lo + at, kRowHi, k_lo + at, kRowHi, idesc, i > 0);
                }
                mma_commit(bar(kSFull + st));
                mma_commit(bar(kEmpty + slot_of(k)));
                if (j + 2 * step >= n) {
                  mma_commit(bar(kQEmpty));
                  if (alone) mma_commit(bar(kQEmpty));
                }
                if (values) mma_commit(bar(kPvDone + st));
              }
              if (values) mma_commit(bar(kEmpty + slot_of(v)));
            }
            __syncwarp();
            issued = true;
            done += values;
          }
        }
        unit += 2 * n;
      }
      if (!ok && lane == 0) fail();
      // The MMAs issued so far read shared memory and write TMEM, which a softmax whose waits ran out would free under
      // them: they end by themselves, so this wait has a limit of its own and not the plan's.
      if (issued) {
        if (elect_one()) mma_commit(bar(kDrain + st));
        __syncwarp();
        const int never = 0;
        wait_phase(bar(kDrain + st), 0, &never, 2000000000ull);
      }
    } else {
      // ---------------------------------------------------------- addresses
      // One warp, four tokens a lane; a tile's pages are looked up before the wait for its place in the ring.
      const int shift = p.page_shift;
      SeqSeg sg;
      sg.ntiles = 0;
      int seg = -1, j = 0;
      for (int it = 0;; ++it) {
        if (++j >= sg.ntiles) {
          ++seg;
          j = 0;
          if (!wait(kSegFull + seg % kSegRing, (seg / kSegRing) & 1)) break;
          sg = segs[seg % kSegRing];
          __syncwarp();
          arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
          if (sg.ntiles == 0) break;
        }
        const int32_t* const table = sg.table_row >= 0 ? p.block_table + static_cast<int64_t>(sg.table_row) * p.bt_stride : nullptr;
        const int64_t head = static_cast<int64_t>(sg.kvh) * p.page_size;
        int32_t in_page[4], page[4];
        bool asked[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t e = (sg.tile0 + j) * kAttnTile + i * 32 + lane;
          asked[i] = e < sg.count;
          page[i] = -1;
          in_page[i] = 0;
          if (asked[i]) {
            const int32_t pos = e < sg.s0 ? e : e + sg.gap;
            const int32_t col = shift >= 0 ? pos >> shift : pos / p.page_size;
            in_page[i] = pos - col * p.page_size;
            if (table) page[i] = table[col];
          }
        }
        const int a = it % kRing;
        if (!wait(kAEmpty + a, (it / kRing + 1) & 1)) break;
        bool bad = false;
        int64_t off[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          off[i] = -1;
          const int at = a * 128 + i * 32 + lane;
          if (page[i] >= 0 && page[i] < p.num_pages) {
            const int64_t vec = head + in_page[i];
            off[i] = (page[i] * p.page_stride + vec * D) * (kE4m3 ? 1 : 2);
            if (kE4m3) {
              const int64_t from = page[i] * p.scale_page_stride + vec;
              cp4(smem_addr(ring_ks + at), p.k_scales + from);
              cp4(smem_addr(ring_vs + at), p.v_scales + from);
            }
          } else {
            if (kE4m3) ring_ks[at] = ring_vs[at] = 1.f;
            bool seen = asked[i];
            const int32_t node = (sg.tile0 + j) * kAttnTile + i * 32 + lane - sg.end0;
            if (seen && p.tree_mask && node >= 0) {  // a drafted token: does a row of the item see it?
              seen = false;
              for (int r = 0; r < sg.nrows && (node >> 5) < p.mask_words; ++r)
                seen |= p.tree_mask[(static_cast<int64_t>(sg.row0) + r) * p.mask_words + (node >> 5)] >> (node & 31) & 1;
            }
            bad |= seen;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ring_off[a * 128 + i * 32 + lane] = off[i];
          const uint32_t mask = __ballot_sync(0xffffffffu, off[i] >= 0);
          if (lane == 0) ring_mask[a * 4 + i] = mask;
        }
        if (kE4m3) {
          cp_arrive(bar(kScFull + a));
          mbar_arrive(bar(kScFull + a));
        }
        if (bad) atomicOr(p.status, kStatusBounds);
        __syncwarp();
        arrive_one(bar(kAFull + a), lane);
      }
      if (!ok && lane == 0) fail();
      cp_wait_all();
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftmaxRegs));
    const int st = (warp - 8) >> 2, quarter = warp & 3;  // stream; this warp's lanes of TMEM
    const int m_row = quarter * 32 + lane;               // this thread's query within its tile
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_col = tmem + lanes + st * 128, o_col = tmem + lanes + 256 + st * D;
    const int my_r = m_row / p.group, my_h = m_row - my_r * p.group;
    bool ok = true;
    auto wait = [&](int b, uint32_t parity) {
      ok = wait_phase(bar(b), parity, abort, limit);
      return ok;
    };
    uint32_t done = 0, other = 0, tile = 0, joins = 0;  // tiles of this stream and of the other; of all; rendezvous of the streams
    for (int seg = 0;; ++seg) {
      if (!wait(kSegFull + seg % kSegRing, (seg / kSegRing) & 1)) break;
      const SeqSeg sg = segs[seg % kSegRing];
      __syncwarp();
      arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
      if (sg.ntiles == 0) break;
      const int first_row = kPair ? st * per_tile : 0;  // of this tile of queries, within the item
      const int rows = min(per_tile, sg.nrows - first_row);
      const bool mine_q = my_r < rows;                  // this thread has a query
      const int my_row = sg.row0 + first_row + my_r;
      const bool any_q = quarter * 32 < rows * p.group;  // a thread of this warp has
      // what all rows of the tile of queries see: [0, all_a) and [all_b, all_c)
      int32_t all_a = 0, all_b = 0, all_c = sg.end0;
      if (!p.tree_mask) {
        int32_t skip;
        row_sees(p, sg, first_row, all_a, skip, all_c);
        row_sees(p, sg, first_row + rows - 1, skip, all_b, skip);
        if (all_b <= all_a) all_b = 0;
      }
      auto scaled = [](float* x, const float* by) {  // kStep tokens' scales
#pragma unroll
        for (int i = 0; i < S::kStep; i += 4) {
          const float4 k = *reinterpret_cast<const float4*>(by + i);
          mul2(x[i], x[i + 1], k.x, k.y);
          mul2(x[i + 2], x[i + 3], k.z, k.w);
        }
      };
      const int step = kPair ? 1 : 2;
      auto unit_of = [&](int j) { return smem_addr(units) + (2 * (tile + j) + 1) % S::kSlots * S::kUnit; };  // tile j's values
      float nm = 0.f, l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;  // running maximum, negated; sum, in four parts
      bool fresh = true;                   // no score above minus infinity so far
      bool far = false;                    // a maximum of this warp's is past kFar; uniform
      if (rows > 0) {
        for (int j = kPair ? 0 : st;; j += step) {
          bool odd = false;  // a value that is not finite, of a token that some row of this warp does not see; uniform
          bool masked = false;  // the tile's scores have been masked, and have their keys' scales
          for (; j < sg.ntiles; j += step) {
            const int a = (tile + j) % kRing;
            if (!kPair && !any_q) {  // nothing to do: what stands in this warp's part of P does not matter
              if (!wait(kSFull + st, done & 1)) break;
              arrive_one(bar(kPFull + st), lane);
              arrive_one(bar(kAEmpty + a), lane);
              ++done;
              continue;
            }
            if (!wait((kE4m3 ? kScFull : kAFull) + a, ((tile + j) / kRing) & 1)) break;  // the tile's mask and scales
            if (!wait(kSFull + st, done & 1)) break;
            tc_fence_after();
            const int32_t e0 = (sg.tile0 + j) * kAttnTile;
            const uint4 there = *reinterpret_cast<const uint4*>(ring_mask + a * 4);
            const bool whole = (there.x & there.y & there.z & there.w) == 0xffffffffu &&
                               ((e0 >= all_b && e0 <= all_c - kAttnTile) || e0 <= all_a - kAttnTile);
            // A tile that some row does not see all of: minus infinity takes the place of a score in TMEM. In a loop, and
            // apart from the common path, as code that is read past costs time too.
            if (__builtin_expect(!whole, 0)) {
              uint32_t hid = 0;  // in lane c, of the 32 tokens from 32 c on those that are there and that some row does not see
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                const uint32_t here = c == 0 ? there.x : c == 1 ? there.y : c == 2 ? there.z : there.w;
                const uint32_t v = mine_q ? here & seen_by(p, sg, e0 + 32 * c, first_row + my_r) : 0u;
                const uint32_t unseen = __reduce_or_sync(0xffffffffu, mine_q ? here & ~v : 0u);
                if (lane == c) hid = unseen;
                float x[32];
                __syncwarp();
                tmem_ld<32>(s_col + 32 * c, x);
                tmem_wait_ld();
                pin<32>(x);
                if (kE4m3) scaled(x, ring_ks + a * 128 + 32 * c);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!((v >> i) & 1)) x[i] = -INFINITY;
                tmem_st32(s_col + 32 * c, x);
              }
              tmem_wait_st();
              if (__any_sync(0xffffffffu, hid != 0)) {
                const uint32_t n = kPair ? tile + j : done;
                if (!wait(full_bar(st, 1, n), full_parity(n))) break;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                  const uint32_t unseen = __shfl_sync(0xffffffffu, hid, c);
                  if (unseen) {
                    bool mine = not_finite<D>(unit_of(j), unseen, 32 * c, lane);
                    if (kE4m3) mine |= ((unseen >> lane) & 1) && !(fabsf(ring_vs[a * 128 + 32 * c + lane]) < INFINITY);
                    odd |= __any_sync(0xffffffffu, mine);
                  }
                }
              }
            }
            constexpr int kStep = S::kStep;  // tokens at a time
            auto load = [&](int c, float* x) {
#pragma unroll
              for (int i = 0; i < kStep; i += 32) tmem_ld<32>(s_col + c + i, x + i);
              float4 by[kE4m3 ? kStep / 4 : 1];  // the scales come while the scores do
              if (kE4m3) {
#pragma unroll
                for (int i = 0; i < kStep / 4; ++i) by[kE4m3 ? i : 0] = *reinterpret_cast<const float4*>(ring_ks + a * 128 + c + 4 * i);
              }
              tmem_wait_ld();
              pin<kStep>(x);
              if (kE4m3 && whole) {
#pragma unroll
                for (int i = 0; i < kStep / 4; ++i) {
                  const float4 k = by[kE4m3 ? i : 0];
                  mul2(x[4 * i], x[4 * i + 1], k.x, k.y);
                  mul2(x[4 * i + 2], x[4 * i + 3], k.z, k.w);
                }
              }
            };
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int c = 0; c < 128; c += kStep) {
              float x[kStep];
              load(c, x);
#pragma unroll
              for (int i = 0; i < kStep; i += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k) top[k] = fmaxf(fmaxf(top[k], x[i + 2 * k]), x[i + 2 * k + 1]);
            }
            float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
            const bool raise = fresh ? most > -INFINITY : most + nm > kTau;
            const bool first = j < step;
            if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
              const float now = raise ? -most : nm, alpha = raise && !fresh ? ex2(now - nm) : 1.f;
              nm = now;
              if (!first && __any_sync(0xffffffffu, raise && !fresh)) {
                l0 *= alpha;
                l1 *= alpha;
                l2 *= alpha;
                l3 *= alpha;
                if (!wait(kPvDone + st, (done - 1) & 1)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 8) {
                  float o[8];
                  tmem_ld<8>(o_col + c, o);
                  tmem_wait_ld();
                  pin<8>(o);
#pragma unroll
                  for (int i = 0; i < 8; ++i) o[i] *= alpha;
                  tmem_st8(o_col + c, o);
                }
              }
              fresh = fresh && !raise;
              far = __any_sync(0xffffffffu, fabsf(nm) > kFar);
            }
            if (__builtin_expect(far, 0)) {
              masked = !whole;
              break;
            }
            // P in bf16, in the place of S: a column for two tokens, behind the reads of those
#pragma unroll 1
            for (int c = 0; c < 128; c += kStep) {
              float x[kStep];
              load(c, x);
              uint32_t w[kStep / 2];
#pragma unroll
              for (int i = 0; i < kStep; i += 4) {
#pragma unroll
                for (int k = i; k < i + 4; k += 2) {
                  fma2(x[k], x[k + 1], p.scale_log2, p.scale_log2, nm, nm);
                  x[k] = ex2(x[k]);
                  x[k + 1] = ex2(x[k + 1]);
                }
                add2(l0, l1, x[i], x[i + 1]);
                add2(l2, l3, x[i + 2], x[i + 3]);
              }
              if (kE4m3) scaled(x, ring_vs + a * 128 + c);
#pragma unroll
              for (int i = 0; i < kStep / 2; ++i) w[i] = bf16x2(x[2 * i], x[2 * i + 1]);
#pragma unroll
              for (int i = 0; i < kStep / 2; i += 16) tmem_st16(s_col + c / 2 + i, w + i);
            }
            tmem_wait_st();
            if (__builtin_expect(odd, 0)) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(kPFull + st));
              mbar_arrive(bar(kAEmpty + a));
            }
            __syncwarp();
            ++done;
          }
          if (!ok || j >= sg.ntiles) break;
          // Rare tiles. Out of the loop over tiles: a call in it, or as much code, costs 16 % of a prefill's time.
          const int a = (tile + j) % kRing, e0 = (sg.tile0 + j) * kAttnTile;
          uint32_t seen[4];
#pragma unroll 1
          for (int c = 0; c < 4; ++c) seen[c] = mine_q ? ring_mask[a * 4 + c] & seen_by(p, sg, e0 + 32 * c, first_row + my_r) : 0u;
          if (far) l0 += far_weights<kE4m3>(s_col, ring_ks + a * 128, ring_vs + a * 128, masked, p.scale_log2, nm);
          if (odd) {
            ok = tile_by_hand<D>(s_col, o_col, unit_of(j), seen, j < step, bar(kPFull + st), bar(kAEmpty + a), bar(kPvDone + st),
                                 done & 1, abort, limit);
            if (!ok) break;
          } else {
            tc_fence_before();
            __syncwarp();
            arrive_one(bar(kPFull + st), lane);
            arrive_one(bar(kAEmpty + a), lane);
          }
          ++done;
        }
      } else if (kPair) {
        // this stream has no queries in the item: its share of the tiles' addresses is free at once
        for (int j = 0; j < sg.ntiles; ++j) {
          if (!wait(kAFull + (tile + j) % kRing, ((tile + j) / kRing) & 1)) break;
          arrive_one(bar(kAEmpty + (tile + j) % kRing), lane);
        }
      }
      if (!ok) break;
      tile += sg.ntiles;
      // ---- the segment's result
      float m = fresh ? kUnset : -nm, l = (l0 + l1) + (l2 + l3);
      float w_own = 1.f, w_other = 0.f;
      constexpr int kCols = kPair ? D : D / 2;  // this thread's columns of the result
      const int col0 = kPair ? 0 : st * kCols;
      const int mine_n = kPair ? sg.ntiles : (sg.ntiles + 1 - st) / 2, other_n = kPair ? 0 : sg.ntiles - mine_n;
      if (rows > 0 && mine_n > 0) {
        if (!wait(kPvDone + st, (done - 1) & 1)) break;
      }
      if (!kPair) {
        other += other_n;
        ml_s[st * 128 + m_row] = make_float2(m, l);
        __syncwarp();
        arrive_one(bar(kJoin), lane);
        if (!wait(kJoin, joins & 1)) break;
        ++joins;
        if (other_n > 0 && !wait(kPvDone + (st ^ 1), (other - 1) & 1)) break;
        const float2 x = ml_s[(st ^ 1) * 128 + m_row];
        const float top = fmaxf(m, x.x);
        w_own = mine_n > 0 ? ex2(m - top) : 0.f;
        w_other = other_n > 0 ? ex2(x.x - top) : 0.f;
        l = (mine_n > 0 ? l * w_own : 0.f) + (other_n > 0 ? x.y * w_other : 0.f);
        m = top;
      }
      if (kPair ? rows > 0 : any_q) {
        tc_fence_after();
        const int64_t head = (static_cast<int64_t>(my_row) * p.kv_heads + sg.kvh) * p.group + my_h;
        const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
        const int m_item = (kPair ? st * 128 : 0) + m_row;
        float* const part = p.part_o + (static_cast<int64_t>(max(sg.slot, 0)) * D + col0) * S::kQueries + m_item;
        uint16_t* const out = p.out + head * D + col0;
#pragma unroll 1
        for (int c = 0; c < kCols; c += 16) {
          float o[16], x[16];
          __syncwarp();
          if (kPair || mine_n > 0) tmem_ld<16>(o_col + col0 + c, o);
          if (!kPair && other_n > 0) tmem_ld<16>(tmem + lanes + 256 + (st ^ 1) * D + col0 + c, x);
          tmem_wait_ld();
          pin<16>(o);
          pin<16>(x);
          if (!kPair) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = (mine_n > 0 ? o[i] * w_own : 0.f) + (other_n > 0 ? x[i] * w_other : 0.f);
          }
          if (sg.slot >= 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * S::kQueries] = o[i];
          } else if (mine_q) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
            *reinterpret_cast<uint4*>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        if (kPair || st == 0) {
          if (sg.slot >= 0)
            p.part_ml[static_cast<int64_t>(sg.slot) * S::kQueries + m_item] = make_float2(m, l);
          else if (p.lse && mine_q)
            p.lse[head] = l == 0.f ? -INFINITY : (m + lg2(l)) * 0.69314718055994531f;
        }
        tc_fence_before();
      }
      if (!kPair) {  // both have read both results before either's next product
        __syncwarp();
        arrive_one(bar(kJoin), lane);
        if (!wait(kJoin, joins & 1)) break;
        ++joins;
      }
    }
    if (!ok && lane == 0) fail();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && abort_flag) atomicOr(p.status, kStatusTimeout);
  if (warp == 5) tmem_dealloc(tmem, S::kTmem);
}

// Join the partials of an item that CTA `first` of the attention kernel began
// and others continued: out = sum_i w_i O_i / sum_i w_i l_i with
// w_i = 2^(m_i - max m), in the order of the list. A block per such item and 32
// queries, a lane each; a warp has every eighth column of the result, or with
// kFew (few such blocks) every eighth partial of 16 columns.
template <int D, int kQueries, bool kFew>
__global__ void __launch_bounds__(256) seq_combine_kernel(const __grid_constant__ SeqAttnParams p, int ctas) {
  constexpr int kCols = kFew ? 16 : D, kPer = kFew ? 16 : D / 8, kWarpParts = kFew ? 8 : 1;
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float o_s[kFew ? 8 : 1][kCols][33];
  __shared__ float2 ml_s[8][32];
  __shared__ int first_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {  // the CTA that began the blockIdx.x-th item that is shared
    int first = -1, seen = 0;
    for (int c = 0; c < ctas && first < 0; c += 32) {
      const uint32_t some = __ballot_sync(0xffffffffu, c + lane < ctas && p.seg_info[c + lane].w > 0);
      const int skip = static_cast<int>(blockIdx.x) - seen;
      seen += __popc(some);
      if (skip < __popc(some)) first = c + static_cast<int>(__fns(some, 0, skip + 1));
    }
    if (lane == 0) first_s = first;
  }
  __syncthreads();
  const int first = first_s;
  if (first < 0) return;
  const int4 info = p.seg_info[first];
  const int parts = info.w + 1, per_tile = 128 / p.group;
  const int m0 = blockIdx.y * 32, mi = m0 + lane, col0 = kFew ? blockIdx.z * kCols : 0;
  auto row_of = [&](int i, int& h) {  // the item's row of query i, -1: none
    const int t = i >> 7, r = (i & 127) / p.group, row = t * per_tile + r;
    h = (i & 127) - r * p.group;
    return r < per_tile && row < info.y ? row : -1;
  };
  int h;
  const bool there = row_of(mi, h) >= 0;
  if (!__syncthreads_or(there)) return;
  auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * first + 1 : 2 * (first + i)); };
  float m = kUnset, l = 0.f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll 2
  for (int i = kFew ? warp : 0; i < parts; i += kWarpParts) {
    const float2 ml = p.part_ml[slot(i) * kQueries + mi];
    float x[kPer];
    const float* const o = p.part_o + (slot(i) * D + col0 + (kFew ? 0 : warp)) * kQueries + mi;
#pragma unroll
    for (int k = 0; k < kPer; ++k) x[k] = o[k * (kFew ? 1 : 8) * kQueries];
    const float now = fmaxf(m, ml.x), old = ex2(m - now), w = ex2(ml.x - now);
    m = now;
    l = l * old + ml.y * w;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = acc[k] * old + x[k] * w;
  }
  if (kFew) {
    ml_s[warp][lane] = make_float2(m, l);
#pragma unroll
    for (int k = 0; k < kPer; ++k) o_s[warp][k][lane] = acc[k];
    __syncthreads();
    m = kUnset;
    l = 0.f;
    for (int w = 0; w < 8; ++w) m = fmaxf(m, ml_s[w][lane].x);
    float sum[kPer / 8] = {};
    for (int w = 0; w < 8; ++w) {
      const float2 ml = ml_s[w][lane];
      const float f = ex2(ml.x - m);
      l += ml.y * f;
#pragma unroll
      for (int k = 0; k < kPer / 8; ++k) sum[k] += o_s[w][warp + 8 * k][lane] * f;
    }
    __syncthreads();
    const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
#pragma unroll
    for (int k = 0; k < kPer / 8; ++k) o_s[0][warp + 8 * k][lane] = sum[k] * inv;
  } else {
    const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
#pragma unroll
    for (int k = 0; k < kPer; ++k) o_s[0][warp + 8 * k][lane] = acc[k] * inv;
  }
  if (p.lse && warp == 0 && there && col0 == 0) {
    const int row = row_of(mi, h);
    p.lse[(static_cast<int64_t>(info.x + row) * p.kv_heads + info.z) * p.group + h] =
        l == 0.f ? -INFINITY : (m + lg2(l)) * 0.69314718055994531f;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 32 * (kCols / 2); e += 256) {
    const int q = e / (kCols / 2), c = e % (kCols / 2) * 2;
    const int row = row_of(m0 + q, h);
    if (row >= 0)
      *reinterpret_cast<uint32_t*>(p.out + ((static_cast<int64_t>(info.x + row) * p.kv_heads + info.z) * p.group + h) * D + col0 + c) =
          bf16x2(o_s[0][c][q], o_s[0][c + 1][q]);
  }
}

namespace {

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Calls f with the kernel of a geometry and its shape.
template <typename F>
cudaError_t with_kernel(int head_dim, bool e4m3, bool pair, F f) {
#define SMQ_SEQ(D, E, P) return f(seq_attention_kernel<D, E, P>, SeqShape<D, E, P>())
#define SMQ_SEQ_STREAMS(D, E) \
  if (pair) SMQ_SEQ(D, E, true); \
  SMQ_SEQ(D, E, false)
  if (head_dim == 128) {
    if (e4m3) {
      SMQ_SEQ_STREAMS(128, true);
    }
    SMQ_SEQ_STREAMS(128, false);
  }
  if (e4m3) {
    SMQ_SEQ_STREAMS(64, true);
  }
  SMQ_SEQ_STREAMS(64, false);
#undef SMQ_SEQ_STREAMS
#undef SMQ_SEQ
}

template <int D, int kQueries>
cudaError_t launch_combine(const SeqAttnParams& p, int grid, cudaStream_t stream) {
  // at most as many items as CTAs are shared, and no more than there are; blocks of 32 queries that some item can have
  const int64_t per = kQueries / 128 * (128 / p.group);
  const int64_t items = (static_cast<int64_t>(p.rows) / per + p.num_seqs) * p.kv_heads;
  const unsigned shared = static_cast<unsigned>(items < grid ? items : grid);
  const unsigned blocks = ((kQueries > 128 ? kQueries : p.max_seq_rows * p.group) + 31) / 32;
  // kFew spreads an item's partials and columns over warps and blocks, which pays as long as there are few blocks of 32 queries:
  // a call in us, kFew and not, 64 heads on 8, D 128: one row of 1, 8, 16 and 64 sequences 20 and 33, 69 and 73, 120 and 122, 221
  // and 223 (8 to 152 blocks); 64 rows of 2, 8 and 16 sequences 58 and 58, 107 and 85, 267 and 244 (384 and 1216 blocks).
  if (shared * blocks <= 2u * static_cast<unsigned>(grid))
    return launch(seq_combine_kernel<D, kQueries, true>, dim3(shared, blocks, D / 16), 256, 0, stream, p, grid);
  return launch(seq_combine_kernel<D, kQueries, false>, dim3(shared, blocks), 256, 0, stream, p, grid);
}

}  // namespace

cudaError_t prepare_seq_attention(int head_dim, bool e4m3) {
  for (int pair = 0; pair < 2; ++pair) {
    const cudaError_t rc = with_kernel(head_dim, e4m3, pair != 0, [](auto kernel, auto shape) {
      // the register split waits for ever on a launch with fewer registers than it hands out
      cudaFuncAttributes a;
      const cudaError_t err = cudaFuncGetAttributes(&a, kernel);
      if (err != cudaSuccess) return err;
      if (a.numRegs != decltype(shape)::kRegs) return cudaErrorInvalidKernelImage;
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, decltype(shape)::kSmem);
    });
    if (rc != cudaSuccess) return rc;
  }
  return cudaSuccess;
}

cudaError_t launch_seq_attention(const SeqAttnParams& p, bool e4m3, int grid, cudaStream_t stream) {
  // Two tiles of queries where some sequence may have more than one: 64 heads on 8, contexts of 8192, 16 sequences of 17 and of 64
  // rows 130 and 244 us, 231 and 440 with one tile; 2 of 1024 rows 416 and 636; 31 of 5 rows, 32 heads on 1, 57 and 80.
  const bool pair = p.max_seq_rows > 128 / p.group;
  cudaError_t rc = with_kernel(p.head_dim, e4m3, pair, [&](auto kernel, auto shape) {
    return launch(kernel, dim3(grid), decltype(shape)::kThreads, decltype(shape)::kSmem, stream, p);
  });
  if (rc != cudaSuccess) return rc;
  if (p.head_dim == 128) return pair ? launch_combine<128, 256>(p, grid, stream) : launch_combine<128, 128>(p, grid, stream);
  return pair ? launch_combine<64, 256>(p, grid, stream) : launch_combine<64, 128>(p, grid, stream);
}

}  // namespace smq
