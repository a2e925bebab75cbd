// Attention of one query row per sequence over the 8-bit cache (q8.cuh):
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(q . k_t / sqrt(128) - max).
//
// Bound by the cache's bytes: 256 per token and KV head, read once for the
// G = nh / nkv query heads that share it. The cache rows go from TMA to the
// tensor core as they are stored, with no conversion: an e4m3 tile of 128
// tokens is the MMA's M operand (kind::mxf8f6f4), once as K (tokens x dims)
// and once as V transposed (dims x tokens). What multiplies them has 8 bits too,
// so q and the probabilities are split into a sum of 8-bit parts:
//   q = 2^e (a1 + a2 / 16 + a3 / 256), e4m3, exact down to 2^-18 of the head's
//       largest element, and to 2^-26 of it below;
//   p = 2^e (a1 + a2 / 8 + a3 / 64), e5m2, to 2^-9 of p (a rounding of 2^-3 in
//       each part), as bf16 would hold it, down to 2^-28 of the largest p that
//       shares the scale; what is smaller, to 2^-37 of that largest.
// Tokens share p's scale 2^e where they share an E8M0 byte of the MMA, 32 tokens
// of a chunk (and the same 32 places of the batch's other chunk): one softmax
// warp, whose maximum is at hand. So the range does not depend on what other
// tokens have: behind a first token of e^16 times the others' probability and a
// small value row, thousands of tiny ones carry the output. (Two e4m3 parts
// under one scale for all tokens, 2^-22 of the largest, lost up to all of it;
// they took 8.7 us at 4096 tokens, 8.9 now, 60 at 131072, 62 now, and the same 56 for
// 32 sequences of 4096.)
// The parts are further columns of the narrow N operand, whose width costs
// nothing: an MMA of 128 x N x 32 takes as long as its 4 KB of M operand do.
// The factors 2^e, 2^-4i, 2^-3i and the scale of the V block are E8M0 scales
// that the tensor core applies; the scale of the K block goes into the softmax's.
//
//   S^T [128 tokens x 3G] = K [128 x 128] . Q^T       O^T [128 dims x 3G] = V^T . P^T
//
// The chunks (128 tokens) of all sequences form one list, cut into equal,
// contiguous parts, so that uneven lengths balance; a part is worked on by nkv
// neighbouring CTAs, one per KV head, which read the same rows of the cache at
// about the same time (two sequences of 131072 and 115000: 91 us, and 124 with
// the heads one after the other in the list).
// A part covers segments of one or more sequences; a segment that is a whole
// sequence is finished in place, another leaves (o, max, sum) in the
// workspace, in one of its CTA's two slots, and a second kernel joins them in
// order (and writes the rows of sequences without tokens). A single sequence is
// balanced as it is: then the up to 16 parts of a head are one cluster, which
// joins them over DSMEM and saves the second launch (512 tokens 6.1 us against
// 7.3, 4096 tokens 9.4, now 8.9, against 10.5, 32768 tokens 20.4 against 22.8;
// and 2.4 us of the host's time). Inside a
// decode call, whose next kernel's weights are on their way meanwhile, the
// clusters gave nothing.
//
// Inside a decode call the token's own row is appended here (k_new): the q warp
// of the CTA that holds a sequence's last chunk stores it by the rule of
// kv_store_q8_kernel, in front of that chunk's loads. (With a store kernel of
// its own: 113.7 us a layer for 32 sequences of 4096 tokens, 110.8 so; 64 of
// 8192 268 and 259.)
//
// Roles per CTA (224 threads, two CTAs per SM): warps 0-3 softmax (thread = token,
// then dimension), warp 4 TMA, warp 5 MMA, warp 6 builds the q parts. Chunks go in
// batches of kBat: the S MMAs of batch j + 1 run while batch j is in the
// softmax, and K tiles are loaded one batch ahead of V tiles.
#include "q3vl_internal.h"
#include "q8.cuh"

namespace q3vl {
namespace {

constexpr int kAqThreads = 224;
constexpr int kAqTiles = 6;               // ring of 16 KB tiles, K and V in turn
constexpr int kAqTile = 128 * 128;
constexpr int kAqRec = 130;               // floats of a head's partial: o[128], max, sum
constexpr int kAqMaxCluster = 16;

template <int G>
struct AqCfg {
  static constexpr int NS = G == 8 ? 32 : 16;      // columns of S and O: 3 G parts
  static constexpr int kBat = 2;                   // chunks per batch
  static constexpr int kQ = NS * 128;              // q parts, e4m3
  // p parts of a chunk, e5m2. G = 8 keeps 24 of its 32 rows: the MMA reads the
  // bytes behind them (the next chunk's, or q's) into columns that no one does.
  static constexpr int kP = (G == 8 ? 24 : 16) * 128;
  // TMEM columns: S of two batches, O, scales of K (ones), q (two segments), V, p
  static constexpr int cS = 0, cO = 2 * kBat * NS, cSfK = cO + NS, cSfQ = cSfK + 4,
                       cSfV = cSfQ + 8, cSfP = cSfV + 4;
  static constexpr uint32_t kCols = G == 8 ? 256 : 128;
  static_assert(cSfP + 4 <= kCols, "TMEM columns");
  static constexpr size_t kSmem = 1024 + size_t(kAqTiles) * kAqTile + size_t(kBat) * kP +
                                  2 * kQ + 2 * 512 + 2 * 4 * 8 * 4 + 4 * 8 * 4 +
                                  (2 * kAqTiles + 9) * 8 + 4 * 2 * 4 + 64;
  static_assert(kSmem <= 115712, "two CTAs per SM");
};

struct AttnQ8Params {
  const __nv_bfloat16* q;   // [B][nh*128]
  uint8_t* kc;              // the cache [n_seq][cap][nkv*128] (written where rows are appended)
  uint8_t* vc;
  uint8_t* ks;              // scales [n_seq][nblk][nkv]
  uint8_t* vs;
  const __nv_bfloat16* k_new;  // [B][nkv*128]: this token's rows, to row len[b]; or null
  const __nv_bfloat16* v_new;
  int64_t cap;
  int n_seq, nblk;
  const int32_t* seq;
  const int32_t* len;
  int plus;                 // tokens attended: len[b] + plus
  int early;                // seq, len and all blocks but each sequence's last are final before the
                            // dependency
  int B, nkv;
  int most;                 // chunks that a slot can hold
  int parts;                // of the chunk list; nkv CTAs each
  int cluster;              // one sequence: the parts of a head are a cluster
  float scale_log2;         // log2(e) / sqrt(128)
  __nv_bfloat16* o;         // [B][nh*128]
  float* part;              // [parts][nkv][2][G][kAqRec]
  int32_t* err;
};

// Chunks of sequence b's tokens (0: none, or out of range).
__device__ __forceinline__ int aq_chunks(const AttnQ8Params& p, int b, bool& ok) {
  const int slot = p.seq[b], L = p.len[b];
  ok = slot >= 0 && slot < p.n_seq && L >= 0 && int64_t(L) + p.plus <= p.cap;
  return ok ? (L + p.plus + 127) / 128 : 0;
}

// A batch: chunks c .. c + nb - 1 of KV head g of sequence b, inside a segment
// [c0, c1) of the sequence's nc chunks.
struct AqBatch {
  int b, g, slot, len, nc, c0, c1, c, nb;
  __device__ bool first() const { return c == c0; }
  __device__ bool last() const { return c + nb == c1; }
};

// Part i of `parts` has chunks [i total / parts, (i + 1) total / parts) of the
// list; there are no more parts than chunks. At most 256 sequences of 1024
// chunks and some hundred parts: the products stay in 32 bits.
__device__ __forceinline__ int aq_parts_of(const AttnQ8Params& p, int total) {
  return min(p.parts, total);
}

// A part's heads are neighbouring CTAs (grid [parts][nkv]); in cluster mode a
// head's parts are (grid [nkv][parts]).
__device__ __forceinline__ int aq_part(const AttnQ8Params& p) {
  return static_cast<int>(p.cluster ? blockIdx.x : blockIdx.y);
}
__device__ __forceinline__ int aq_head(const AttnQ8Params& p) {
  return static_cast<int>(p.cluster ? blockIdx.y : blockIdx.x);
}

// Chunks of the sequences of one lane, 8 l .. 8 l + 7, and how many come before
// them. Every role's warp makes its own: no barrier stands between the lengths
// and the first load.
struct AqList {
  uint32_t n[4];            // two counts (<= 1024) to a word
  int base, total;
  int u0, u1;               // this CTA's part of the list
  __device__ AqList(const AttnQ8Params& p, int lane, bool report) {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int b = 8 * lane + i;
      bool ok = true;
      const int k = b < p.B ? aq_chunks(p, b, ok) : 0;
      if (!ok && report) record_error(p.err, Q3VL_ERANGE, kWhereAttnQ8Range);
      sum += k;
      n[i / 2] = i & 1 ? n[i / 2] | (uint32_t(k) << 16) : uint32_t(k);
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    base = inc - sum;
    total = __shfl_sync(0xffffffffu, inc, 31);
    const int part = aq_part(p), parts = aq_parts_of(p, total);
    u0 = u1 = 0;
    if (part < parts) {
      u0 = static_cast<int>(static_cast<uint32_t>(total * part) / static_cast<uint32_t>(parts));
      u1 = static_cast<int>(static_cast<uint32_t>(total * (part + 1)) / static_cast<uint32_t>(parts));
    }
  }
  // The sequence that chunk u of the list belongs to (whole warp).
  __device__ void find(int u, int& b, int& start, int& nc) const {
    int at = base, hit = -1, k = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = (n[i / 2] >> (16 * (i & 1))) & 0xffff;
      if (u >= at && u < at + c) { hit = i; start = at; k = c; }
      at += c;
    }
    const int lane = threadIdx.x & 31;
    const int src = __ffs(__ballot_sync(0xffffffffu, hit >= 0)) - 1;
    b = __shfl_sync(0xffffffffu, 8 * lane + hit, src);
    start = __shfl_sync(0xffffffffu, start, src);
    nc = __shfl_sync(0xffffffffu, k, src);
  }
};

// The batches of this CTA's part of the chunk list (whole warps).
template <int kBat>
struct AqIter {
  const AttnQ8Params& p;
  const AqList& list;
  int u, u1;
  AqBatch t{};
  __device__ AqIter(const AttnQ8Params& p_, const AqList& l) : p(p_), list(l), u(l.u0), u1(l.u1) {
    t.g = aq_head(p);
  }
  __device__ bool next(AqBatch& out) {
    if (t.c + t.nb < t.c1) {
      t.c += t.nb;
    } else {
      if (u >= u1) return false;
      int start = 0;
      list.find(u, t.b, start, t.nc);
      t.c0 = u - start;
      t.c1 = min(t.c0 + u1 - u, t.nc);
      u += t.c1 - t.c0;
      t.c = t.c0;
      t.slot = p.seq[t.b];
      t.len = p.len[t.b] + p.plus;
    }
    t.nb = min(kBat, t.c1 - t.c);
    out = t;
    return true;
  }
};

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %1, %1, %1};" ::"r"(taddr), "r"(w)
               : "memory");
}
// e for probabilities 2^(s - M) of scores up to `top` <= M: the largest lies in
// [2^e, 2^(e + 1)). At least -96, far below what fp32 sums keep and above the
// end of the E8M0 bytes; also where there is no score (top = -inf) or M is NaN.
__device__ __forceinline__ float aq_p_exponent(float top, float M) {
  return fmaxf(floorf(top - M), -96.f);
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.sync 1, 128;" ::: "memory"); }

// Registers: two CTAs per SM, and for up to four heads enough left beside them
// for two blocks of the joining kernel, which then starts before this one ends
// (4 sequences of 4096 tokens 14.5 us, and 16.9 with 118 registers).
template <int G, bool APPEND>
__global__ void __maxnreg__(G == 8 ? 128 : 112)
attn_q8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               AttnQ8Params p) {
  using C = AqCfg<G>;
  constexpr int NS = C::NS, kBat = C::kBat;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* s_tile = smem;                                  // [kAqTiles][128 x 128]
  uint8_t* s_p = s_tile + kAqTiles * kAqTile;              // [kBat][16 x 128]
  uint8_t* s_q = s_p + kBat * C::kP;                       // [2][NS x 128]
  uint8_t* s_qs = s_q + 2 * C::kQ;                         // [2][512] scale words of the q parts
  uint64_t* full = reinterpret_cast<uint64_t*>(s_qs + 2 * 512);
  uint64_t* empty = full + kAqTiles;
  uint64_t* s_full = empty + kAqTiles;                     // [2]
  uint64_t* q_full = s_full + 2;                           // [2]
  uint64_t* q_empty = q_full + 2;                          // [2]
  uint64_t* p_full = q_empty + 2;
  uint64_t* o_full = p_full + 1;
  uint64_t* drain = o_full + 1;
  float* s_wm = reinterpret_cast<float*>(drain + 1);      // [2][4 warps][8] maxima
  float* s_wl = s_wm + 2 * 4 * 8;                          // [4 warps][8] sums
  uint32_t* s_sc = reinterpret_cast<uint32_t*>(s_wl + 4 * 8);  // [4][2] scales of appended-to blocks
  uint32_t* tmem_slot = s_sc + 4 * 2;
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) {
    for (int i = 0; i < kAqTiles; ++i) { mbar_init(full + i, 1); mbar_init(empty + i, 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1); mbar_init(q_full + i, 1); mbar_init(q_empty + i, 1);
    }
    mbar_init(p_full, 4);
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  if (warp < 4) {
    // p parts of the columns from 3 G on stay zero
    for (int i = t; i < kBat * C::kP / 16; i += 128)
      *reinterpret_cast<uint4*>(s_p + 16 * i) = make_uint4(0, 0, 0, 0);
  } else if (warp == 6) {
    for (int i = lane; i < 2 * C::kQ / 16; i += 32)
      *reinterpret_cast<uint4*>(s_q + 16 * i) = make_uint4(0, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();  // behind the allocation: no later grid's can come before it
  const uint32_t lf = static_cast<uint32_t>((warp & 3) * 32) << 16;
  if (warp < 4) {
    tmem_st4(tmem + lf + C::cSfK, kNoScale);  // constant scales: ones for K
    tmem_st_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // lengths and slots are inputs of the call, not of the kernel before
  if (!APPEND) griddep_wait();
  const AqList list(p, lane, blockIdx.x == 0 && blockIdx.y == 0 && warp == 4);
  if (APPEND && (warp < 4 || warp == 6)) griddep_wait();
  if (warp == 4) {
    AqIter<kBat> ik(p, list), iv(p, list);
    AqBatch bk, bv;
    int stage = 0, issued = 0, seg = -1;
    uint32_t ph = 1;
    bool ok = true;
    auto load = [&](const AqBatch& a, const CUtensorMap* tm, bool keys) {
      if (keys && a.first()) ++seg;
      for (int i = 0; i < a.nb && ok; ++i) {
        // the block that the q warp appends to (V's tiles come behind K's)
        if (APPEND && keys && a.c + i == a.nc - 1)
          ok = __all_sync(0xffffffffu, mbar_wait(q_full + (seg & 1), (seg >> 1) & 1, p.err,
                                                 kWhereAttnQ8, s_abort));
        if (!ok) break;
        ok = __all_sync(0xffffffffu, mbar_wait(empty + stage, ph, p.err, kWhereAttnQ8, s_abort));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(full + stage, kAqTile);
          tma_load_2d(s_tile + stage * kAqTile, tm, full + stage, a.g * 128,
                      static_cast<int32_t>(int64_t(a.slot) * p.cap + int64_t(a.c + i) * 128));
        }
        __syncwarp();
        ++issued;
        if (++stage == kAqTiles) { stage = 0; ph ^= 1; }
      }
    };
    if (ik.next(bk)) load(bk, &tmK, true);
    while (ok && iv.next(bv)) {
      if (ik.next(bk)) load(bk, &tmK, true);
      if (ok) load(bv, &tmV, false);
    }
    // every issued load lands before the CTA may exit
    for (int i = issued > kAqTiles ? issued - kAqTiles : 0; i < issued; ++i)
      mbar_wait(full + i % kAqTiles, (i / kAqTiles) & 1, p.err, kWhereAttnQ8, nullptr);
  } else if (warp == 5) {
    constexpr uint32_t id_s = idesc_mxf8(128, NS);
    constexpr uint32_t id_o = idesc_mxf8(128, NS) | (1u << 10) | (1u << 15);  // p e5m2, V transposed
    AqIter<kBat> is(p, list), iv(p, list);
    AqBatch bs, bv;
    int stage = 0, js = 0, jv = 0, seg = 0;
    uint32_t ph = 0;
    bool ok = true;
    auto step = [&]() { if (++stage == kAqTiles) { stage = 0; ph ^= 1; } };
    auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, p.err, kWhereAttnQ8, s_abort));
    };
    auto scores = [&](const AqBatch& a) {
      const int qb = seg & 1;
      const uint32_t sfq = tmem + C::cSfQ + 4 * qb;
      if (a.first()) {
        ok = wait(q_full + qb, (seg >> 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t ds = sdesc_scales(smem_u32(s_qs + qb * 512));
        if (elect_one()) tmem_cp_scales(sfq, ds);
        __syncwarp();
      }
      const uint64_t dq = sdesc_sw128(smem_u32(s_q + qb * C::kQ), 16, 1024);
      for (int i = 0; i < a.nb; ++i) {
        ok = wait(full + stage, ph);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dk = sdesc_sw128(smem_u32(s_tile + stage * kAqTile), 16, 1024);
        const uint32_t d = tmem + C::cS + ((js & 1) * kBat + i) * NS;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_mxf8_ss(d, dk + 2 * kk, dq + 2 * kk, id_s, tmem + C::cSfK, sfq, kk > 0 ? 1u : 0u);
          umma_commit(empty + stage);
        }
        __syncwarp();
        step();
      }
      if (elect_one()) {
        umma_commit(s_full + (js & 1));
        if (a.last()) umma_commit(q_empty + qb);
      }
      __syncwarp();
      ++js;
      if (a.last()) ++seg;
    };
    if (is.next(bs)) scores(bs);
    while (ok && iv.next(bv)) {
      if (is.next(bs)) scores(bs);
      if (!ok || !wait(p_full, jv & 1)) break;
      tc_fence_after();
      for (int i = 0; i < bv.nb; ++i) {
        ok = wait(full + stage, ph);
        if (!ok) break;
        tc_fence_after();
        uint8_t* v = s_tile + stage * kAqTile;
        const int rows = bv.len - (bv.c + i) * 128;
        if (rows < 128) {
          // rows behind the sequence hold whatever the cache had: zero, for
          // 0 * NaN would not be
          for (int k = rows * 8 + lane; k < 128 * 8; k += 32)
            *reinterpret_cast<uint4*>(v + 16 * k) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t dv = sdesc_sw128(smem_u32(v), 16, 1024);
        const uint64_t dp = sdesc_sw128(smem_u32(s_p + i * C::kP), 16, 1024);
        const uint32_t id = id_o | (static_cast<uint32_t>(i) << 29);  // V's scale: byte i
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // p's scale: byte kk
            umma_mxf8_ss(tmem + C::cO, dv + 256 * kk, dp + 2 * kk,
                         id | (static_cast<uint32_t>(kk) << 4), tmem + C::cSfV, tmem + C::cSfP,
                         (i | kk) > 0 ? 1u : 0u);
          umma_commit(empty + stage);
          if (i == bv.nb - 1) umma_commit(o_full);
        }
        __syncwarp();
        step();
      }
      ++jv;
    }
    if (!ok) *s_abort = 1;
    // all issued MMAs complete before the TMEM is released
    if (elect_one()) umma_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, p.err, kWhereAttnQ8, nullptr);
  } else if (warp == 6) {
    // q parts: row n = part * G + h of the N operand, and its scale
    AqIter<kBat> it(p, list);
    AqBatch a;
    int seg = 0;
    // this token's K and V rows into row len - 1 of the sequence, 4 elements a
    // lane; the scales of their blocks to sc
    auto append = [&](const AqBatch& e, uint32_t* sc) {
      const int row = e.len - 1, blk = row >> 7;
      const int64_t si = (int64_t(e.slot) * p.nblk + blk) * p.nkv + e.g, rs = int64_t(p.nkv) * 128;
      const int64_t ni = (int64_t(e.b) * p.nkv + e.g) * 128 + 4 * lane;
      const bool keeps = (row & 127) != 0;  // the block holds earlier rows
      if (!dcheck(e.slot < p.n_seq && row < p.cap, p.err, kWhereDbgQ8)) return;
      const uint2 now[2] = {*reinterpret_cast<const uint2*>(p.k_new + ni),
                            *reinterpret_cast<const uint2*>(p.v_new + ni)};
      const uint32_t old[2] = {keeps ? p.ks[si] : 0u, keeps ? p.vs[si] : 0u};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = unpack_bf16x2(now[i].x), y = unpack_bf16x2(now[i].y);
        uint32_t u = e8m0_of_amax(redux_max(fmaxf(fmaxf(finite_abs(x.x), finite_abs(x.y)),
                                                  fmaxf(finite_abs(y.x), finite_abs(y.y)))));
        const uint32_t was = old[i];
        if (keeps && was >= u) u = was;
        uint8_t* dst = (i == 0 ? p.kc : p.vc) + int64_t(e.slot) * p.cap * rs + e.g * 128 + 4 * lane;
        if (keeps && u > was) {
          const float m = u - was > 126 ? 0.f : e8m0_inverse(127 + (u - was));
#pragma unroll 4
          for (int r = blk * 128; r < row; ++r) {
            uint32_t* w = reinterpret_cast<uint32_t*>(dst + r * rs);
            const float4 f = unpack_e4m3x4(*w);
            *w = pack_e4m3x4(f.x * m, f.y * m, f.z * m, f.w * m);
          }
        }
        const float s = e8m0_inverse(u);
        *reinterpret_cast<uint32_t*>(dst + row * rs) = pack_e4m3x4(x.x * s, x.y * s, y.x * s, y.y * s);
        if (lane == 0) {
          (i == 0 ? p.ks : p.vs)[si] = static_cast<uint8_t>(u);
          sc[i] = u;
        }
      }
      // the tile's loads go through the async proxy
      __threadfence();
      asm volatile("fence.proxy.async;" ::: "memory");
    };
    while (it.next(a)) {
      if (!a.first()) continue;
      const int qb = seg & 1;
      if (seg >= 2 &&
          !__all_sync(0xffffffffu, mbar_wait(q_empty + qb, ((seg >> 1) - 1) & 1, p.err,
                                             kWhereAttnQ8, s_abort)))
        break;
      const __nv_bfloat16* src = p.q + (int64_t(a.b) * p.nkv + a.g) * G * 128 + 4 * lane;
      uint2 raw[G];
#pragma unroll
      for (int h = 0; h < G; ++h) raw[h] = *reinterpret_cast<const uint2*>(src + h * 128);
      if (APPEND && a.c1 == a.nc) append(a, s_sc + 2 * (seg & 3));
      uint32_t word = kNoScale;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float2 x = unpack_bf16x2(raw[h].x), y = unpack_bf16x2(raw[h].y);
        float f[4] = {x.x, x.y, y.x, y.y};
        const float am = redux_max(fmaxf(fmaxf(finite_abs(f[0]), finite_abs(f[1])),
                                         fmaxf(finite_abs(f[2]), finite_abs(f[3]))));
        const uint32_t e = max(e8m0_of_amax(am), 16u);  // room for the parts' smaller scales
        const float inv = e8m0_inverse(e);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] *= inv;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const int n = part * G + h;
          const uint32_t w = pack_e4m3x4(f[0], f[1], f[2], f[3]);
          const float4 r = unpack_e4m3x4(w);
          f[0] = (f[0] - r.x) * 16.f; f[1] = (f[1] - r.y) * 16.f;
          f[2] = (f[2] - r.z) * 16.f; f[3] = (f[3] - r.w) * 16.f;
          *reinterpret_cast<uint32_t*>(s_q + qb * C::kQ + n * 128 +
                                       (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4) = w;
          if (lane == n) word = (e - 4 * part) * 0x01010101u;
        }
      }
      *reinterpret_cast<uint4*>(s_qs + qb * 512 + lane * 16) =
          make_uint4(word, kNoScale, kNoScale, kNoScale);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + qb);
      ++seg;
    }
  } else {
    // A wait that gives up raises s_abort, which makes every later one return
    // at once: these warps then walk through the rest without results, so that
    // all four pass the same named barriers.
    AqIter<kBat> it(p, list);
    AqBatch a;
    int j = 0, seg = -1;
    float* rec = reinterpret_cast<float*>(s_tile);  // this CTA's record, once the ring is done
    if (p.cluster && it.u >= it.u1) {  // no chunks: an empty record
#pragma unroll
      for (int h = 0; h < G; ++h) {
        rec[h * kAqRec + t] = 0.f;
        if (t == 0) { rec[h * kAqRec + 128] = -INFINITY; rec[h * kAqRec + 129] = 0.f; }
      }
    }
    float m_run[G], l_run[G], o_run[G], fade[G];
    // this lane's word of p's scales: row `lane` of the N operand is part
    // lane / G of head lane % G; m_lane is that head's running maximum
    const int row_part = lane / G, row_head = lane % G;
    float m_lane = -INFINITY;
    while (it.next(a)) {
      if (a.first()) {
        ++seg;
        m_lane = -INFINITY;
#pragma unroll
        for (int h = 0; h < G; ++h) { m_run[h] = -INFINITY; l_run[h] = o_run[h] = fade[h] = 0.f; }
      }
      // scales of the batch's blocks, requested ahead of the scores
      const int64_t si = (int64_t(a.slot) * p.nblk + a.c) * p.nkv + a.g;
      uint8_t kb[kBat], vb[kBat];
#pragma unroll
      for (int i = 0; i < kBat; ++i) {
        const int64_t at = si + int64_t(min(i, a.nb - 1)) * p.nkv;
        const bool appended = APPEND && a.c + i >= a.nc - 1;
        kb[i] = appended ? 127 : p.ks[at];
        vb[i] = appended ? 127 : p.vs[at];
      }
      mbar_wait(s_full + (j & 1), (j >> 1) & 1, p.err, kWhereAttnQ8, s_abort);
      __syncwarp();
      tc_fence_after();
      // the q warp left them before the q parts of these scores; it comes back
      // to the slot four segments on, behind products of two segments on, which
      // wait for this batch
      if (APPEND)
#pragma unroll
        for (int i = 0; i < kBat; ++i)
          if (a.c + i == a.nc - 1) {
            kb[i] = static_cast<uint8_t>(s_sc[2 * (seg & 3)]);
            vb[i] = static_cast<uint8_t>(s_sc[2 * (seg & 3) + 1]);
          }
      float sc[kBat][G];
#pragma unroll
      for (int i = 0; i < kBat; ++i) {
        uint32_t u[NS];
        if (i < a.nb) {
          const uint32_t at = tmem + lf + C::cS + ((j & 1) * kBat + i) * NS;
          if constexpr (NS == 16) tmem_ld16(at, u);
          else tmem_ld32(at, u);
          tmem_ld_wait();
        }
        const bool sees = i < a.nb && (a.c + i) * 128 + t < a.len;
        const float f = e8m0_scale(kb[i]) * p.scale_log2;
#pragma unroll
        for (int h = 0; h < G; ++h)
          sc[i][h] = sees ? ((__uint_as_float(u[h]) + __uint_as_float(u[G + h])) +
                             __uint_as_float(u[2 * G + h])) * f
                          : -INFINITY;
      }
      float* wm = s_wm + (j & 1) * 32;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float v = sc[0][h];
#pragma unroll
        for (int i = 1; i < kBat; ++i) v = fmaxf(v, sc[i][h]);
        v = redux_max(v);
        if (lane == 0) wm[warp * 8 + h] = v;
      }
      softmax_sync();
      float next_fade[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float M = fmaxf(fmaxf(fmaxf(wm[h], wm[8 + h]), fmaxf(wm[16 + h], wm[24 + h])),
                              m_run[h]);
        next_fade[h] = ex2_approx(m_run[h] - M);
        m_run[h] = M;
        // 2^(e + 14) holds this warp's largest p, so p is 2^e times at most 2^15.
        // The sums carry a factor 2^8, which the quotient drops.
        const float e = aq_p_exponent(wm[warp * 8 + h], M);
        float l = 0.f;
#pragma unroll
        for (int i = 0; i < kBat; ++i) {
          sc[i][h] = ex2_approx((sc[i][h] - M) + (14.f - e));
          l += sc[i][h];
        }
        l_run[h] = fmaf(l, __uint_as_float(static_cast<uint32_t>(int(e) + 127 + 8 - 14) << 23),
                        l_run[h] * next_fade[h]);
      }
      m_lane = fmaxf(fmaxf(fmaxf(wm[row_head], wm[8 + row_head]),
                           fmaxf(wm[16 + row_head], wm[24 + row_head])), m_lane);
      uint32_t pw = 0;  // byte w: the scale of the tokens of warp w
#pragma unroll
      for (int w = 0; w < 4; ++w)
        pw |= static_cast<uint32_t>(int(aq_p_exponent(wm[8 * w + row_head], m_lane)) + 127 + 8 -
                                    14 - 3 * row_part) << (8 * w);
      // the batch before: its products, behind which P and V's scales are free
      auto fold = [&](int of) {
        mbar_wait(o_full, of & 1, p.err, kWhereAttnQ8, s_abort);
        __syncwarp();
        tc_fence_after();
        uint32_t u[NS];
        if constexpr (NS == 16) tmem_ld16(tmem + lf + C::cO, u);
        else tmem_ld32(tmem + lf + C::cO, u);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < G; ++h)
          o_run[h] = o_run[h] * fade[h] + ((__uint_as_float(u[h]) + __uint_as_float(u[G + h])) +
                                           __uint_as_float(u[2 * G + h]));
      };
      if (!a.first()) fold(j - 1);
#pragma unroll
      for (int h = 0; h < G; ++h) fade[h] = next_fade[h];
      uint32_t vw = 0;
#pragma unroll
      for (int i = 0; i < kBat; ++i) vw |= uint32_t(vb[i]) << (8 * i);
      tmem_st4(tmem + lf + C::cSfV, vw);
      tmem_st4(tmem + lf + C::cSfP, row_part < 3 ? pw : kNoScale);
#pragma unroll
      for (int i = 0; i < kBat; ++i) {
        if (i >= a.nb) break;
        uint8_t* dst = s_p + i * C::kP + (t & 15);
        float v[(G + 3) / 4 * 4];
#pragma unroll
        for (int h = 0; h < (G + 3) / 4 * 4; ++h) v[h] = h < G ? sc[i][h < G ? h : 0] : 0.f;
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int h0 = 0; h0 < G; h0 += 4) {
            const uint32_t w = pack_e5m2x4(v[h0], v[h0 + 1], v[h0 + 2], v[h0 + 3]);
            if (part < 2) {
              const float4 r = unpack_e5m2x4(w);
              v[h0] = (v[h0] - r.x) * 8.f; v[h0 + 1] = (v[h0 + 1] - r.y) * 8.f;
              v[h0 + 2] = (v[h0 + 2] - r.z) * 8.f; v[h0 + 3] = (v[h0 + 3] - r.w) * 8.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (h0 + k < G) {
                const int n = part * G + h0 + k;
                dst[n * 128 + (((t >> 4) ^ (n & 7)) << 4)] = static_cast<uint8_t>(w >> (8 * k));
              }
          }
      }
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
      if (a.last()) {
        fold(j);
        tc_fence_before();
        // the sum over the threads' tokens
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float l = warp_sum(l_run[h]);
          if (lane == 0) s_wl[warp * 8 + h] = l;
        }
        softmax_sync();
        const bool whole = !p.cluster && a.c0 == 0 && a.c1 == a.nc;
        __nv_bfloat16* ob = p.o + (int64_t(a.b) * p.nkv + a.g) * G * 128 + t;
        float* pb = p.cluster ? rec
                              : p.part + ((int64_t(blockIdx.y) * p.nkv + a.g) * 2 + (a.c0 == 0 ? 1 : 0)) * G *
                                             kAqRec;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float l = (s_wl[h] + s_wl[8 + h]) + (s_wl[16 + h] + s_wl[24 + h]);
          if (whole) {
            ob[h * 128] = __float2bfloat16_rn(o_run[h] / l);
          } else {
            pb[h * kAqRec + t] = o_run[h];
            if (t == 0) { pb[h * kAqRec + 128] = m_run[h]; pb[h * kAqRec + 129] = l; }
          }
        }
        softmax_sync();  // s_wl is free
      }
      ++j;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if (p.cluster) {
    cluster_sync();  // every CTA's record is in its shared memory
    if (t < 128) {
      const int g = blockIdx.y;
      for (int i = static_cast<int>(cluster_ctarank()) * 128 + t; i < G * 128; i += p.parts * 128) {
        const int h = i >> 7, d = i & 127;
        const uint32_t own = smem_u32(s_tile) + h * kAqRec * 4;
        // all records requested before any is used
        float m[kAqMaxCluster], l[kAqMaxCluster], o[kAqMaxCluster], M = -INFINITY;
#pragma unroll
        for (int k = 0; k < kAqMaxCluster; ++k) {
          const uint32_t at = map_to_cta(own, static_cast<uint32_t>(k < p.parts ? k : 0));
          m[k] = k < p.parts ? ld_dsmem_f32(at + 128 * 4) : -INFINITY;
          l[k] = k < p.parts ? ld_dsmem_f32(at + 129 * 4) : 0.f;
          o[k] = k < p.parts ? ld_dsmem_f32(at + 4 * d) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAqMaxCluster; ++k) M = fmaxf(M, m[k]);
        float num = 0.f, den = 0.f;
#pragma unroll
        for (int k = 0; k < kAqMaxCluster; ++k) {
          if (l[k] == 0.f) continue;  // empty
          const float w = ex2_approx(m[k] - M);
          num = fmaf(w, o[k], num);
          den = fmaf(w, l[k], den);
        }
        // no tokens at all: zeros
        p.o[(int64_t(g) * G + h) * 128 + d] = __float2bfloat16_rn(den == 0.f ? 0.f : num / den);
      }
    }
    cluster_sync();  // no record leaves while another CTA may read it
  }
}

// Joins the segments of the sequences that more than one part holds, in the
// order of their chunks:
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  M = max_s m_s,
// and writes zeros where there are no tokens. One block per sequence and query
// head, of 128 threads, or of four groups of 128 that share out the segments
// where there can be many of them (one sequence of 20000 tokens and 2 KV heads,
// 148 segments: 17.3 us, and 21.5 with one group); the weights of all segments are made at once, thread =
// segment, then thread = dimension.
constexpr int kAqMaxParts = 512;

template <int kGroups>
__global__ void __launch_bounds__(128 * kGroups) attn_q8_join_kernel(AttnQ8Params p, int G) {
  constexpr int kThreads = 128 * kGroups, kWarps = 4 * kGroups;
  __shared__ int s_i[2][kWarps];
  __shared__ float s_f[2][kWarps];
  __shared__ float s_w[kAqMaxParts];
  __shared__ float s_o[kGroups][128];
  const int t = threadIdx.x, nh = G * p.nkv, b = blockIdx.x / nh, qh = blockIdx.x % nh;
  const int g = qh / G, h = qh % G, warp = t >> 5, lane = t & 31, d = t & 127, grp = t >> 7;
  griddep_launch_dependents();
  if (!p.early) griddep_wait();
  // chunks before b, and of all
  int before = 0, total = 0;
  bool ok;
  for (int i = t; i < p.B; i += kThreads) {
    const int n = aq_chunks(p, i, ok);
    total += n;
    before += i < b ? n : 0;
  }
  const int nc = aq_chunks(p, b, ok);
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) { s_i[0][warp] = before; s_i[1][warp] = total; }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) { before += s_i[0][i]; total += s_i[1][i]; }
  const int parts = aq_parts_of(p, total);
  int i0 = 0, n = 0;  // parts i0 .. i0 + n - 1
  if (nc > 0) {
    i0 = static_cast<int>(static_cast<uint32_t>((before + 1) * parts - 1) / static_cast<uint32_t>(total));
    n = static_cast<int>(static_cast<uint32_t>((before + nc) * parts - 1) /
                         static_cast<uint32_t>(total)) - i0 + 1;
  }
  if (p.early) griddep_wait();
  __nv_bfloat16* out = p.o + int64_t(blockIdx.x) * 128 + d;
  if (nc == 0 && grp == 0) *out = __float2bfloat16_rn(0.f);
  if (n <= 1) return;  // finished in place
  // part i's record: its second slot where the sequence starts in it
  auto rec = [&](int s) {
    return p.part + ((int64_t(i0 + s) * p.nkv + g) * 2 + (s == 0 ? 1 : 0)) * G * kAqRec + h * kAqRec;
  };
  // this group's segments: grp, grp + kGroups, ..., kU of them requested at a time
  constexpr int kU = 16;
  float o[kU];
  auto request = [&](int s0) {
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int s = s0 + k * kGroups + grp;
      o[k] = s < n ? __ldcg(rec(s) + d) : 0.f;
    }
  };
  request(0);
  constexpr int kEach = kAqMaxParts / kThreads;
  float m[kEach], l[kEach], M = -INFINITY;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int s = t + kThreads * k;
    m[k] = s < n ? __ldcg(rec(s) + 128) : -INFINITY;
    l[k] = s < n ? __ldcg(rec(s) + 129) : 0.f;
    M = fmaxf(M, m[k]);
  }
  M = warp_max(M);
  if (lane == 0) s_f[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, s_f[0][i]);
  float den = 0.f;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int s = t + kThreads * k;
    const float w = s < n ? ex2_approx(m[k] - M) : 0.f;
    s_w[s] = w;
    if (s < n) den = fmaf(w, l[k], den);
  }
  den = warp_sum(den);
  if (lane == 0) s_f[1][warp] = den;
  __syncthreads();
  den = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) den += s_f[1][i];
  float num = 0.f;
  for (int s0 = 0; s0 < n; s0 += kU * kGroups) {
    if (s0 > 0) request(s0);
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int s = s0 + k * kGroups + grp;
      if (s < n) num = fmaf(s_w[s], o[k], num);
    }
  }
  if (kGroups > 1) {
    s_o[grp][d] = num;
    __syncthreads();
    if (grp > 0) return;
    num = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) num += s_o[i][d];
  }
  *out = __float2bfloat16_rn(num / den);
}

// Two CTAs per SM, and no more parts than there can be chunks.
int aq_parts(int nkv, int B, int64_t cap) {
  const int64_t most = int64_t(B) * ((cap + 127) / 128);
  int64_t parts = 2 * sm_count() / nkv > 1 ? 2 * sm_count() / nkv : 1;
  if (parts > kAqMaxParts) parts = kAqMaxParts;
  return static_cast<int>(most < parts ? most : parts);
}

template <int G>
cudaError_t launch_g(const CUtensorMap& tmK, const CUtensorMap& tmV, AttnQ8Params p,
                     cudaStream_t st) {
  auto kern = p.k_new != nullptr ? attn_q8_kernel<G, true> : attn_q8_kernel<G, false>;
  cudaError_t e = smem_attr_at_least(reinterpret_cast<const void*>(kern), AqCfg<G>::kSmem);
  if (e != cudaSuccess) return e;
  if (p.B == 1 && p.k_new == nullptr) {
    // up to 16 parts of each head while two CTAs per SM hold them all, if that is
    // not far fewer than the list would have
    const void* fn = reinterpret_cast<const void*>(kern);
    int cs = 2 * sm_count() / p.nkv, n = 0;
    if (cs > kAqMaxCluster) cs = kAqMaxCluster;
    if (cs > p.most) cs = p.most;
    if (cs >= 1 && 3 * cs >= (p.most < p.parts ? p.most : p.parts)) {
      e = allow_nonportable_clusters(fn);
      if (e == cudaSuccess)
        e = max_active_clusters(fn, kAqThreads, AqCfg<G>::kSmem, cs, &n);
      if (e != cudaSuccess) return e;
    }
    if (n >= 1) {
      p.cluster = 1;
      p.parts = cs;
      e = launch_pdl_cluster(kern, dim3(cs, p.nkv), dim3(kAqThreads), AqCfg<G>::kSmem, st, cs, tmK,
                             tmV, p);
      return e != cudaSuccess ? e : counted_launch(1);
    }
  }
  e = launch_pdl_plain(kern, dim3(p.nkv, p.parts), dim3(kAqThreads), AqCfg<G>::kSmem, st, tmK, tmV,
                       p);
  if (e != cudaSuccess) return e;
  const dim3 rows(p.B * p.nkv * G);
  e = p.parts > 48 ? launch_pdl_plain(attn_q8_join_kernel<4>, rows, dim3(512), 0, st, p, G)
                   : launch_pdl_plain(attn_q8_join_kernel<1>, rows, dim3(128), 0, st, p, G);
  return e != cudaSuccess ? e : counted_launch(2);
}

}  // namespace

size_t attention_q8_ws_bytes(const q3vl_config& c, int B, int64_t cap) {
  const int G = c.n_heads / c.n_kv_heads;
  return align256(size_t(aq_parts(c.n_kv_heads, B, cap)) * c.n_kv_heads * 2 * G * kAqRec * sizeof(float));
}

cudaError_t launch_attention_q8(const q3vl_config& c, const void* q, int B,
                                const q3vl_kv_cache_q8& kv, const int32_t* seq,
                                const int32_t* len, const void* k_new, const void* v_new, void* o,
                                void* ws, cudaStream_t st) {
  const uint64_t rows = uint64_t(kv.n_seq) * uint64_t(kv.cap), dkv = uint64_t(kv_dim(c));
  CUtensorMap tmK, tmV;
  if (!make_tmap_u8(&tmK, kv.k, rows, dkv, dkv, 128, 128) ||
      !make_tmap_u8(&tmV, kv.v, rows, dkv, dkv, 128, 128))
    return cudaErrorInvalidValue;
  AttnQ8Params p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kc = kv.k; p.vc = kv.v; p.ks = kv.k_scale; p.vs = kv.v_scale;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.cap = kv.cap; p.n_seq = kv.n_seq; p.nblk = static_cast<int>((kv.cap + 127) / 128);
  p.seq = seq; p.len = len;
  p.plus = p.early = k_new != nullptr ? 1 : 0;
  p.B = B; p.nkv = c.n_kv_heads;
  p.parts = aq_parts(c.n_kv_heads, B, kv.cap);
  p.most = p.nblk;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / 11.313708498984761);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.part = static_cast<float*>(ws);
  p.err = device_error_ptr();
  const int G = c.n_heads / c.n_kv_heads;
  switch (G) {
    case 1: return launch_g<1>(tmK, tmV, p, st);
    case 2: return launch_g<2>(tmK, tmV, p, st);
    case 4: return launch_g<4>(tmK, tmV, p, st);
    case 8: return launch_g<8>(tmK, tmV, p, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace q3vl
