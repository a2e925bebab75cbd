// Product of 8-bit rows and an 8-bit weight with block scales (q8.cuh):
//   out[m][n] = sum_j 2^(xs[m][j] + ws[n / 128][j] - 254) sum_{k in block j} xq[m][k] wq[n][k]
// (+ resid[m][n]), summed in fp32 and rounded once.
//
// The tensor core multiplies e4m3 at twice the bf16 rate and, because the
// scales are powers of two, applies them itself (tcgen05.mma kind::mxf8f6f4,
// one scale byte per operand row and 32 columns, here the same byte for the
// four steps of a 128-column block). The partial sums of one output therefore
// stay in one fp32 accumulator over the whole of K, and splitting K needs no
// more than an addition. TMA brings the operand tiles (128-byte swizzle, 128
// columns a box); a warp builds the scale words in the layout that the tensor
// core reads (q8.cuh), each with the bytes of four k-blocks, and the MMA
// thread copies them to TMEM once per four k-blocks. (A word per k-block, the
// first form, cost 200 against 187 us at 4096 x 2560 x 19456: the copies hold
// up the MMAs behind them.)
#include "q3vl_internal.h"
#include "q8.cuh"

namespace q3vl {
namespace {

constexpr int kKB = 128;                // k-block: bytes of K per stage and scale
constexpr int kScaleBytes = 512;        // scale words of 128 rows, four k-blocks
constexpr int kSG = 4;                  // k-blocks per scale word

struct LinQ8Params {
  int64_t M, N;
  int kblk;                // k-blocks: ceil(K / 128)
  const uint8_t* xs;       // [M][kblk]
  const uint8_t* ws;       // [ceil(N / 128)][kblk]
  bool words;              // rows of xs and ws are whole, aligned 32-bit words
  const void* resid;       // [M][N] or null
  void* out;               // [M][N]
  int32_t* err;
};

__device__ __forceinline__ void add4(const __nv_bfloat16* r, float (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(r);
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
  v[0] += a.x; v[1] += a.y; v[2] += b.x; v[3] += b.y;
}
__device__ __forceinline__ void add4(const float* r, float (&v)[4]) {
  const float4 u = *reinterpret_cast<const float4*>(r);
  v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
}
__device__ __forceinline__ void put4(__nv_bfloat16* o, const float (&v)[4]) {
  __stcs(reinterpret_cast<uint2*>(o), make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])));
}
__device__ __forceinline__ void put4(float* o, const float (&v)[4]) {
  __stcs(reinterpret_cast<float4*>(o), make_float4(v[0], v[1], v[2], v[3]));
}

// 32 bytes of a row (32-byte aligned): a whole sector from one thread.
__device__ __forceinline__ void put32(void* o, const uint32_t (&w)[8]) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void get32(const void* i, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(i)
               : "memory");
}

// 32 columns of one output row from n (a multiple of 32), for rows whose
// 32-byte units are whole and aligned.
__device__ __forceinline__ void finish_wide(const LinQ8Params& p, int64_t m, int64_t n,
                                            const float (&v)[32], __nv_bfloat16*) {
  const int64_t at = m * p.N + n;
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    if (n + i >= p.N) return;
    uint32_t w[8], r[8];
    if (p.resid != nullptr) get32(static_cast<const __nv_bfloat16*>(p.resid) + at + i, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float2 f = make_float2(v[i + 2 * j], v[i + 2 * j + 1]);
      if (p.resid != nullptr) {
        const float2 q = unpack_bf16x2(r[j]);
        f.x += q.x; f.y += q.y;
      }
      w[j] = pack_bf16x2(f.x, f.y);
    }
    put32(static_cast<__nv_bfloat16*>(p.out) + at + i, w);
  }
}
__device__ __forceinline__ void finish_wide(const LinQ8Params& p, int64_t m, int64_t n,
                                            const float (&v)[32], float*) {
  const int64_t at = m * p.N + n;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    if (n + i >= p.N) return;
    uint32_t w[8], r[8];
    if (p.resid != nullptr) get32(static_cast<const float*>(p.resid) + at + i, r);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = __float_as_uint(v[i + j] + (p.resid != nullptr ? __uint_as_float(r[j]) : 0.f));
    put32(static_cast<float*>(p.out) + at + i, w);
  }
}

// Four neighbouring columns n .. n + 3 of output row m (n a multiple of 4):
// the residual and the rounding. Rows of a width that is no multiple of 4
// start anywhere, so they go element by element.
template <typename T>
__device__ __forceinline__ void finish4(const LinQ8Params& p, int64_t m, int64_t n, float (&v)[4]) {
  if (!dcheck(m < p.M, p.err, kWhereDbgQ8)) return;
  const int64_t at = m * p.N + n;
  T* o = static_cast<T*>(p.out) + at;
  const T* r = static_cast<const T*>(p.resid) + at;
  if ((p.N & 3) == 0) {
    if (n >= p.N) return;
    if (p.resid != nullptr) add4(r, v);
    put4(o, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N)
        o[i] = static_cast<T>(v[i] + (p.resid != nullptr ? static_cast<float>(r[i]) : 0.f));
  }
}

// Scale bytes k .. k + 3 of a row of `end` bytes as one word (the last byte
// repeated behind the end). `words`: rows are whole, aligned words, as for
// every K that is a multiple of 512; else four loads, which cost the warp that
// makes the words four times the load instructions. Coherent loads: the kernel
// may be resident while the one before it writes these bytes.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int k, int end, bool words) {
  if (words && k + kSG <= end) return *reinterpret_cast<const uint32_t*>(row + k);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < kSG; ++i) w |= uint32_t(row[min(k + i, end - 1)]) << (8 * i);
  return w;
}

// ---------------------------------------------------------------------------
// Few rows: the weight is the MMA's M operand (128 rows a tile) and a tile of
// NB <= 128 rows of x its N operand, so that one decoded token pads N to 16
// and not M to 128. Bound by the weight's bytes; K is split over up to 8 CTAs
// of a cluster (about two CTAs per SM stream weights), which leave their fp32
// partial tiles in shared memory and share out the rows of x to add them up
// over DSMEM in split order: the sum has one order whatever the timing.
// ---------------------------------------------------------------------------
constexpr int kSkThreads = 192;         // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue, 2 scales first
constexpr int kSkMaxSplits = 8;         // portable cluster size
constexpr int kSkMaxNB = 128;           // scale words of one copy; 224 measured 24.8 against 16.9 us at
                                        // 256 x 9728 x 2560: half the CTAs, a ring half as deep

struct SkSched {
  int NB = 16, ttiles = 1, tiles = 1, splits = 1, stages = 2;
  uint32_t tcols = 32;
  size_t smem = 0;
};

template <typename T>
__global__ void __launch_bounds__(kSkThreads, 2)
linear_q8_rows_kernel(const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmX, LinQ8Params p, SkSched sc) {
  constexpr uint32_t kABytes = 128 * kKB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int S = sc.stages;
  const uint32_t b_bytes = static_cast<uint32_t>(sc.NB) * kKB;   // a multiple of 2 KB
  uint8_t* smA = smem;
  uint8_t* smB = smA + size_t(S) * kABytes;
  uint8_t* smS = smB + size_t(S) * b_bytes;                       // [2]: weight, x
  uint64_t* full = reinterpret_cast<uint64_t*>(smS + 4 * kScaleBytes);
  uint64_t* empty = full + S;
  uint64_t* sfull = empty + S;
  uint64_t* sempty = sfull + 2;
  uint64_t* acc_full = sempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = static_cast<int>(blockIdx.x) % sc.splits;
  const int tt = static_cast<int>(blockIdx.x) / sc.splits % sc.ttiles;
  const int tile = static_cast<int>(blockIdx.x) / sc.splits / sc.ttiles;
  const int k_lo = static_cast<int>(int64_t(split) * p.kblk / sc.splits);
  const int n = static_cast<int>(int64_t(split + 1) * p.kblk / sc.splits) - k_lo;
  const int64_t m0 = int64_t(tt) * sc.NB;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full + s, 1); mbar_init(empty + s, 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(sfull + s, 1); mbar_init(sempty + s, 1); }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, sc.tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();

  if (warp == 0) {
    const int32_t row0 = tile * 128;
    const int pre = n < S ? n : S;
    // the weights may be asked for ahead of the dependency, as far as L2
    if (elect_one())
      for (int i = 0; i < pre; ++i) tma_prefetch_2d(&tmW, (k_lo + i) * kKB, row0);
    griddep_wait();
    int issued = 0, s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < n; ++i) {
      if (!mbar_wait(empty + s, ph, p.err, kWhereLinearQ8, abort_flag)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(full + s, kABytes + b_bytes);
        tma_load_2d(smA + size_t(s) * kABytes, &tmW, full + s, (k_lo + i) * kKB, row0);
        tma_load_2d(smB + size_t(s) * b_bytes, &tmX, full + s, (k_lo + i) * kKB,
                    static_cast<int32_t>(m0));
      }
      __syncwarp();
      issued = i + 1;
      if (++s == S) { s = 0; ph ^= 1; }
    }
    // every issued load lands before the CTA may exit
    for (int i = issued - S > 0 ? issued - S : 0; i < issued; ++i)
      mbar_wait(full + (i % S), (i / S) & 1, p.err, kWhereLinearQ8, nullptr);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_mxf8(128, sc.NB);
    bool ok = true;
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n; ++i) {
      const int g = i / kSG;
      const bool fresh = i % kSG == 0;
      // two sets of scale columns in turn, behind the accumulator
      const uint32_t sfa = tmem_base + sc.NB + (g & 1) * 8, sfx = sfa + 4;
      ok = !fresh || mbar_wait(sfull + (g & 1), (g >> 1) & 1, p.err, kWhereLinearQ8, abort_flag);
      ok = ok && mbar_wait(full + s, ph, p.err, kWhereLinearQ8, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint64_t da = sdesc_sw128(smem_u32(smA + size_t(s) * kABytes), 16, 1024);
      const uint64_t db = sdesc_sw128(smem_u32(smB + size_t(s) * b_bytes), 16, 1024);
      const uint64_t ds = sdesc_scales(smem_u32(smS + (g & 1) * 2 * kScaleBytes));
      const uint32_t id = idesc | idesc_sf(i % kSG);
      if (elect_one()) {
        if (fresh) {
          tmem_cp_scales(sfa, ds);
          tmem_cp_scales(sfx, ds + kScaleBytes / 16);
          umma_commit(sempty + (g & 1));
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_mxf8_ss(tmem_base, da + 2 * kk, db + 2 * kk, id, sfa, sfx, (i | kk) != 0 ? 1u : 0u);
        umma_commit(empty + s);
        if (i == n - 1) umma_commit(acc_full);
      }
      __syncwarp();
      if (++s == S) { s = 0; ph ^= 1; }
    }
    if (!ok) *abort_flag = 1;
  } else {
    griddep_wait();
    if (warp == 2) {
      // Scale words: the bytes of four k-blocks for the weight tile and for
      // each row of x (rows past M are zero: any scale), requested one group
      // ahead of the one being written.
      const int groups = (n + kSG - 1) / kSG;
      uint32_t x[4], w, nx[4], nw;
      const bool words = p.words && k_lo % kSG == 0;
      auto request = [&](int g) {
        const int k = k_lo + g * kSG, end = k_lo + n;
        nw = scale_word(p.ws + int64_t(tile) * p.kblk, k, end, words);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = lane + 32 * j;
          nx[j] = r < sc.NB && m0 + r < p.M
                      ? scale_word(p.xs + (m0 + r) * p.kblk, k, end, words) : kNoScale;
        }
      };
      request(0);
      for (int g = 0; g < groups; ++g) {
        w = nw;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = nx[j];
        bool ok = true;
        if (g >= 2) {
          if (lane == 0)
            ok = mbar_wait(sempty + (g & 1), ((g >> 1) - 1) & 1, p.err, kWhereLinearQ8, abort_flag);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        if (!ok) break;
        uint8_t* dst = smS + (g & 1) * 2 * kScaleBytes + lane * 16;
        *reinterpret_cast<uint4*>(dst) = make_uint4(w, w, w, w);
        *reinterpret_cast<uint4*>(dst + kScaleBytes) = make_uint4(x[0], x[1], x[2], x[3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull + (g & 1));
        if (g + 1 < groups) request(g + 1);  // behind the fence, which would wait for it
      }
    }
    __syncwarp();
    // TMEM lanes 32 q .. 32 q + 31 of warp q = warp % 4 are this tile's weight
    // rows, columns are rows of x
    bool ok = true;
    if (lane == 0) ok = mbar_wait(acc_full, 0, p.err, kWhereLinearQ8, abort_flag);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    if (!ok) *abort_flag = 1;
  }
  // Split sum over the cluster. Each CTA leaves its fp32 partial tile, [row of
  // x][128], in its own (drained) stage ring; after a cluster barrier CTA
  // `split` finishes rows j = split (mod splits). Every thread of every CTA of
  // the cluster passes the same cluster barriers.
  static_assert(kSkMaxNB <= 128, "a tile has to fit in the ring");
  // S >= 2 stages of 128 (128 + NB) bytes hold NB rows of 512: NB <= 128
  __syncthreads();  // all roles done: loads landed, MMAs committed or abandoned
  const bool run = *abort_flag == 0;
  tc_fence_after();
  float* red = reinterpret_cast<float*>(smem);
  const int rows = static_cast<int>(p.M - m0 < sc.NB ? p.M - m0 : sc.NB);
  if (warp >= 2 && run) {
    const int q = warp & 3;
    const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll 1
    for (int c0 = 0; c0 < rows; c0 += 16) {
      uint32_t u[16];
      tmem_ld16(tb + c0, u);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (c0 + c < rows) red[(c0 + c) * 128 + 32 * q + lane] = __uint_as_float(u[c]);
    }
  }
  // TMEM goes back before any CTA waits for another: a CTA that held it at the
  // cluster barrier could keep out, on its SM, one of another cluster, a peer of
  // which in turn keeps out the CTA that it waits for (products of two streams).
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, sc.tcols);
  }
  cluster_sync();  // every CTA's partials are in its shared memory
  if (warp >= 2 && run) {
#pragma unroll 1
    for (int jj = split + (warp - 2) * sc.splits; jj < rows; jj += 8 * sc.splits) {
      // two rows at a time, every split's values requested before any is
      // added: one DSMEM round trip, then the sum in split order
      const int j1 = jj + 4 * sc.splits;
      float4 w[2][kSkMaxSplits];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t own = smem_u32(red + (i == 0 || j1 >= rows ? jj : j1) * 128 + 4 * lane);
#pragma unroll
        for (int sp = 0; sp < kSkMaxSplits; ++sp)
          if (sp < sc.splits) w[i][sp] = ld_dsmem_f32x4(map_to_cta(own, sp));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int sp = 0; sp < kSkMaxSplits; ++sp)
          if (sp < sc.splits) {
            v[0] += w[i][sp].x; v[1] += w[i][sp].y; v[2] += w[i][sp].z; v[3] += w[i][sp].w;
          }
        const int j = i == 0 ? jj : j1;
        if (j < rows) finish4<T>(p, m0 + j, int64_t(tile) * 128 + 4 * lane, v);
      }
    }
  }
  cluster_sync();  // no CTA leaves its buffer while another may read it
}

// ---------------------------------------------------------------------------
// Many rows: x is the M operand of a CTA pair (tcgen05.mma cta_group::2, a
// 256 x BN tile, each CTA staging its 128 rows of x and BN / 2 rows of the
// weight per k-block), persistent over tiles, bound by the tensor cores. Two
// accumulators let the epilogue of a tile overlap the next tile's products;
// TMEM holds them and two sets of scale columns (of one CTA: 128 rows of x and
// the tile's BN weight rows), so BN is at most 224, not 256. Shared memory is
// as busy as the tensor core (per k-block 30 KB written by TMA and 30 KB read by
// the MMAs in 448 cycles of 128 bytes), so the epilogue stays out of it where
// rows allow: each thread stores whole 32-byte sectors of its own row. Measured
// at 4096 x 2560 x 19456: 150 us (2700 TFLOP/s), 168 with the stores coalesced
// through shared memory in fp32, 155 with TMA stores of rounded boxes.
// ---------------------------------------------------------------------------
constexpr int kPairThreads = 256;       // warp 0 TMA, 1 MMA, 2-5 epilogue, 6-7 scales
constexpr int kEpiLd = 36;              // floats per row of a warp's 32 x 32 staging block

template <int BN, bool WIDE>
struct PairCfg {
  static constexpr int kABytes = 128 * kKB;
  static constexpr int kBBytes = BN / 2 * kKB;
  static constexpr int kStages = 6;                // 7 measured no faster
  static constexpr int kScales = 3 * kScaleBytes;  // x rows; weight rows 0-127, 128-255
  static constexpr int kSlots = 4;                 // of scale words, two for each of its warps
  static constexpr int kEpi = WIDE ? 0 : 4 * 32 * kEpiLd * 4;
  static constexpr int kAcc = (BN + 31) / 32 * 32;
  static constexpr int kSfCol = 2 * kAcc;          // two sets of 12 columns
  static constexpr size_t kSmem =
      1024 + size_t(kStages) * (kABytes + kBBytes) + size_t(kSlots) * kScales + kEpi + 256;
  static_assert(BN % 32 == 0 && kBBytes % 1024 == 0, "MMA and swizzle");
  static_assert(BN > 128 && BN <= 256, "scale words of two times 128 weight rows");
  static_assert(kSfCol + 24 <= 512, "TMEM columns");
  static_assert(kSmem <= 232448, "shared memory");
};

template <typename T, int BN, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
linear_q8_pair_kernel(const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ CUtensorMap tmW, LinQ8Params p, int tiles_m,
                      int tiles) {
  using C = PairCfg<BN, WIDE>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* smA = smem;
  uint8_t* smB = smA + S * C::kABytes;
  uint8_t* smS = smB + S * C::kBBytes;
  float* smE = reinterpret_cast<float*>(smS + C::kSlots * C::kScales);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(smE) + C::kEpi);
  uint64_t* empty = full + S;
  uint64_t* sfull = empty + S;
  uint64_t* sempty = sfull + C::kSlots;
  uint64_t* tfull = sempty + C::kSlots;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool lead = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    // of the even CTA, full: its TMA thread, whose bytes count both CTAs'
    // loads; sfull: both scale warps; tempty: both CTAs' four epilogue warps
    for (int s = 0; s < S; ++s) { mbar_init(full + s, 1); mbar_init(empty + s, 1); }
    for (int s = 0; s < C::kSlots; ++s) { mbar_init(sfull + s, 2); mbar_init(sempty + s, 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(tfull + b, 1); mbar_init(tempty + b, 8); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();

  if (warp == 0) {
    griddep_wait();
    int stage = 0;
    uint32_t ph = 0, issued = 0, last_ph = 0;  // the latter two: a bit per stage
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += pairs) {
      const int32_t m0 = (t % tiles_m) * 256 + static_cast<int32_t>(rank) * 128;
      const int32_t n0 = (t / tiles_m) * BN + static_cast<int32_t>(rank) * (BN / 2);
      for (int kb = 0; kb < p.kblk; ++kb) {
        ok = mbar_wait<true>(empty + stage, ph ^ 1, p.err, kWhereLinearQ8, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t fb = map_to_cta(smem_u32(full + stage), 0);
          if (lead) mbar_arrive_expect_tx(full + stage, 2 * (C::kABytes + C::kBBytes));
          tma_load_2d_pair(smA + stage * C::kABytes, &tmX, fb, kb * kKB, m0);
          tma_load_2d_pair(smB + stage * C::kBBytes, &tmW, fb, kb * kKB, n0);
        }
        __syncwarp();
        issued |= 1u << stage;
        last_ph = (last_ph & ~(1u << stage)) | (ph << stage);
        if (++stage == S) { stage = 0; ph ^= 1; }
      }
    }
    // every issued load lands before the pair exits (the even CTA's barrier
    // counts both CTAs' bytes; the last cluster barrier holds the odd CTA)
    if (lead)
      for (int s = 0; s < S; ++s)
        if (issued & (1u << s))
          mbar_wait<true>(full + s, (last_ph >> s) & 1u, p.err, kWhereLinearQ8, nullptr);
  } else if (warp == 1) {
    if (lead) {
      constexpr uint32_t idesc = idesc_mxf8(256, BN);
      int stage = 0, it = 0, slot = 0, set = 1;
      uint32_t ph = 0, sph = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs, ++it) {
        const int buf = it & 1;
        ok = mbar_wait<true>(tempty + buf, ((it >> 1) & 1) ^ 1, p.err, kWhereLinearQ8, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * C::kAcc;
        for (int kb = 0; kb < p.kblk; ++kb) {
          const bool fresh = kb % kSG == 0;
          ok = !fresh || mbar_wait<true>(sfull + slot, sph, p.err, kWhereLinearQ8, abort_flag);
          ok = ok && mbar_wait<true>(full + stage, ph, p.err, kWhereLinearQ8, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (fresh) set ^= 1;
          const uint32_t sfx = tmem_base + C::kSfCol + set * 12, sfw = sfx + 4;
          const uint64_t da = sdesc_sw128(smem_u32(smA + stage * C::kABytes), 16, 1024);
          const uint64_t db = sdesc_sw128(smem_u32(smB + stage * C::kBBytes), 16, 1024);
          const uint64_t ds = sdesc_scales(smem_u32(smS + slot * C::kScales));
          const uint32_t id = idesc | idesc_sf(kb % kSG);
          if (elect_one()) {
            if (fresh) {
              tmem_cp_scales_pair(sfx, ds);
              tmem_cp_scales_pair(sfw, ds + kScaleBytes / 16);
              tmem_cp_scales_pair(sfw + 4, ds + 2 * (kScaleBytes / 16));
              umma_commit_pair(sempty + slot, 0x3);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_mxf8_ss_pair(d, da + 2 * k, db + 2 * k, id, sfx, sfw, (kb | k) != 0 ? 1u : 0u);
            umma_commit_pair(empty + stage, 0x3);
            if (kb == p.kblk - 1) umma_commit_pair(tfull + buf, 0x3);
          }
          __syncwarp();
          if (fresh && ++slot == C::kSlots) { slot = 0; sph ^= 1; }
          if (++stage == S) { stage = 0; ph ^= 1; }
        }
      }
      if (elect_one()) umma_commit_pair(drain, 0x3);
      __syncwarp();
    }
  } else if (warp >= 6) {
    griddep_wait();
    // Scale words: the bytes of four k-blocks for each row of x (lane's rows
    // lane + 32 j; rows past M are zero: any scale) and each weight row, whose
    // tile touches up to three 128-row blocks. The two warps take the groups
    // of four k-blocks in turn: one group (0.9 us of MMAs) is not much more
    // than the latency of its loads and of the proxy fence.
    const int half = warp - 6;
    int slot = half;
    uint32_t ph = 0;
    bool ok = true;
    const int wblks = static_cast<int>((p.N + 127) / 128), groups = (p.kblk + kSG - 1) / kSG;
    uint32_t nx[4], nw[3];
    auto request = [&](int t, int g) {
      const int64_t m0 = int64_t(t % tiles_m) * 256 + rank * 128;
      const int w0 = (t / tiles_m) * BN / 128;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = m0 + lane + 32 * j;
        nx[j] = r < p.M ? scale_word(p.xs + r * p.kblk, g * kSG, p.kblk, p.words) : kNoScale;
      }
#pragma unroll
      for (int j = 0; j < 3; ++j)
        nw[j] = scale_word(p.ws + int64_t(min(w0 + j, wblks - 1)) * p.kblk, g * kSG, p.kblk,
                           p.words);
    };
    // this warp's groups: every second one of the sequence over all tiles
    int t = pair, g = half;
    auto settle = [&]() {
      while (g >= groups && t < tiles) { g -= groups; t += pairs; }
    };
    settle();
    if (t < tiles) request(t, g);
    while (t < tiles) {
      const int n0 = (t / tiles_m) * BN, w0 = n0 / 128;
      uint32_t x[4], w[3], u[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = nx[j];
#pragma unroll
      for (int j = 0; j < 3; ++j) w[j] = nw[j];
      if (lane == 0)
        ok = mbar_wait<true>(sempty + slot, ph ^ 1, p.err, kWhereLinearQ8, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      uint8_t* dst = smS + slot * C::kScales + lane * 16;
      *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int b = (n0 + lane + 32 * j) / 128 - w0;  // 0 .. 2
        u[j] = b == 0 ? w[0] : b == 1 ? w[1] : w[2];
      }
      *reinterpret_cast<uint4*>(dst + kScaleBytes) = make_uint4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<uint4*>(dst + 2 * kScaleBytes) = make_uint4(u[4], u[5], u[6], u[7]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_peer(map_to_cta(smem_u32(sfull + slot), 0));
      slot ^= 2;
      if (slot == half) ph ^= 1;
      g += 2;
      settle();
      if (t < tiles) request(t, g);  // behind the fence, which would wait for it
    }
    __syncwarp();
  } else {
    griddep_wait();
    const int q = warp & 3;
    float* se = smE + (warp - 2) * 32 * kEpiLd;
    const uint32_t lane_field = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t tempty_lead = map_to_cta(smem_u32(tempty), 0);
    int it = 0;
    for (int t = pair; t < tiles; t += pairs, ++it) {
      const int buf = it & 1;
      const int64_t m0 = int64_t(t % tiles_m) * 256 + rank * 128 + 32 * q;
      const int64_t n0 = int64_t(t / tiles_m) * BN;
      bool ok = true;
      if (lane == 0)
        ok = mbar_wait<true>(tfull + buf, (it >> 1) & 1, p.err, kWhereLinearQ8, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + buf * C::kAcc + lane_field;
#pragma unroll 1
      for (int cc = 0; cc < BN / 32; ++cc) {
        uint32_t u[32];
        tmem_ld32(tb + 32 * cc, u);
        tmem_ld_wait();
        if (cc == BN / 32 - 1) {  // the accumulator is read: hand it back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_peer(tempty_lead + buf * sizeof(uint64_t));
        }
        if constexpr (WIDE) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
          if (m0 + lane < p.M)
            finish_wide(p, m0 + lane, n0 + 32 * cc, v, static_cast<T*>(nullptr));
        } else {
          // through shared memory, so that a row's 32 columns leave together
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(se + lane * kEpiLd + 4 * j) =
                make_float4(__uint_as_float(u[4 * j]), __uint_as_float(u[4 * j + 1]),
                            __uint_as_float(u[4 * j + 2]), __uint_as_float(u[4 * j + 3]));
          __syncwarp();
          const int64_t n = n0 + 32 * cc + lane;
          const int rows = static_cast<int>(p.M - m0 < 32 ? p.M - m0 : 32);
          if (n < p.N)
#pragma unroll 8
            for (int r = 0; r < rows; ++r) {
              const int64_t at = (m0 + r) * p.N + n;
              float v = se[r * kEpiLd + lane];
              if (p.resid != nullptr) v += static_cast<float>(static_cast<const T*>(p.resid)[at]);
              static_cast<T*>(p.out)[at] = static_cast<T>(v);
            }
          __syncwarp();
        }
      }
    }
  }
  // All issued MMAs complete before either CTA releases its TMEM. Behind the
  // other roles: warp 1 of the odd CTA has no loop, and a wait from the start
  // would have the time limit of one step for the whole product.
  __syncthreads();
  if (warp == 1) mbar_wait<true>(drain, 0, p.err, kWhereLinearQ8, nullptr);
  tc_fence_before();
  cluster_sync();  // no CTA of the pair leaves while the other may touch its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <typename T, int BN, bool WIDE>
cudaError_t launch_pair(const uint8_t* xq, int64_t M, const uint8_t* wq, int64_t N, int64_t K,
                        const LinQ8Params& p, cudaStream_t st) {
  using C = PairCfg<BN, WIDE>;
  CUtensorMap tmX, tmW;
  if (!make_tmap_u8(&tmX, xq, M, K, K, kKB, 128) || !make_tmap_u8(&tmW, wq, N, K, K, kKB, BN / 2))
    return cudaErrorInvalidValue;
  const int64_t tiles_m = (M + 255) / 256, tiles = tiles_m * ((N + BN - 1) / BN);
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  auto kern = linear_q8_pair_kernel<T, BN, WIDE>;
  cudaError_t e = smem_attr_at_least(reinterpret_cast<const void*>(kern), C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = tiles < sm_count() / 2 ? tiles : sm_count() / 2;
  e = launch_pdl_plain(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(kPairThreads), C::kSmem,
                       st, tmX, tmW, p, static_cast<int>(tiles_m), static_cast<int>(tiles));
  if (e != cudaSuccess) return e;
  return counted_launch(1);
}

SkSched sk_sched(int64_t M, int64_t N, int64_t K) {
  SkSched s;
  s.ttiles = static_cast<int>((M + kSkMaxNB - 1) / kSkMaxNB);
  s.NB = static_cast<int>(((M + s.ttiles - 1) / s.ttiles + 15) / 16 * 16);
  s.tiles = static_cast<int>((N + 127) / 128);
  const int kblk = static_cast<int>((K + kKB - 1) / kKB);
  const size_t stage = size_t(128) * kKB + size_t(s.NB) * kKB;
  while (s.tcols < static_cast<uint32_t>(s.NB + 16)) s.tcols <<= 1;
  const int64_t work = int64_t(s.tiles) * s.ttiles;
  int64_t splits = 2 * int64_t(sm_count()) / work;
  if (splits > kSkMaxSplits) splits = kSkMaxSplits;
  if (splits > kblk) splits = kblk;
  // every tile's cluster inside one GPC (16 SMs counted of each) in the first wave
  const int gpcs = sm_count() / 18 > 1 ? sm_count() / 18 : 1;
  while (splits > 1 && (32 / splits) * gpcs < work) --splits;
  s.splits = static_cast<int>(splits < 1 ? 1 : splits);
  // a ring that leaves room for a second CTA on the SM, this kernel's or the
  // next one's, no deeper than the work (200 KB where there is one CTA per SM
  // kept the next launch out: 14.5 us against 8.5 in a row of 1 x 9728 x 2560,
  // split seven ways so)
  const int most = (kblk + s.splits - 1) / s.splits;
  int st = static_cast<int>(size_t(108 * 1024) / stage);
  st = st < 2 ? 2 : (st > 8 ? 8 : st);
  s.stages = st > most ? (most < 2 ? 2 : most) : st;
  s.smem = 1024 + size_t(s.stages) * stage + size_t(4) * kScaleBytes +
           size_t(2 * s.stages + 5) * 8 + 16;
  return s;
}

template <typename T>
cudaError_t launch_rows(const uint8_t* xq, int64_t M, const uint8_t* wq, int64_t N, int64_t K,
                        const LinQ8Params& p, const SkSched& s, cudaStream_t st) {
  CUtensorMap tmW, tmX;
  if (!make_tmap_u8(&tmW, wq, N, K, K, kKB, 128) || !make_tmap_u8(&tmX, xq, M, K, K, kKB, s.NB))
    return cudaErrorInvalidValue;
  const int64_t grid = int64_t(s.tiles) * s.ttiles * s.splits;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  auto kern = linear_q8_rows_kernel<T>;
  cudaError_t e = smem_attr_at_least(reinterpret_cast<const void*>(kern), s.smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl_cluster(kern, dim3(static_cast<unsigned>(grid)), dim3(kSkThreads), s.smem, st,
                         s.splits, tmW, tmX, p, s);
  if (e != cudaSuccess) return e;
  return counted_launch(1);
}

// About how long the two kernels take, in us, fitted to both over M = 1 .. 4096
// at the decoder's weights. Rows: the split sum grows with the width of x's
// tile, a k-block of a CTA costs its MMAs and scales or its CTAs' share of HBM.
// Pair: a start, then all of K for each wave of tiles. Measured rows / pair:
// 1 x 9728 x 2560 8.6 / 25.2, 512 x 9728 x 2560 20.9 / 26.4, 1024 x 9728 x 2560
// 37.8 / 28.2, 128 x 2560 x 6144 11.9 / 12.5, 256 x 2560 x 6144 14.0 / 11.9,
// 64 x 2560 x 19456 15.3 / 17.5, 128 x 2560 x 19456 19.6 / 18.0,
// 4 x 2560 x 151936 65 / 95.
double rows_us(const SkSched& s, int kblk) {
  const double ctas = double(s.tiles) * s.ttiles * s.splits, slots = 2.0 * sm_count();
  const double waves = ctas > slots ? ctas / slots : 1.0, busy = ctas < slots ? ctas : slots;
  const double mma = 0.15 + 0.0025 * s.NB, hbm = 0.0025 * busy;
  return 5.5 + 0.035 * s.NB +
         waves * ((kblk + s.splits - 1) / s.splits) * (mma > hbm ? mma : hbm);
}
double pair_us(int64_t M, int64_t N, int kblk) {
  const int64_t tiles = ((M + 255) / 256) * ((N + 223) / 224), pairs = sm_count() / 2;
  const int64_t waves = (tiles + pairs - 1) / pairs;
  const double mma = 5.2 + 0.26 * double(waves) * (kblk + 4), hbm = 6 + 2e-5 * double(N) * kblk;
  return mma > hbm ? mma : hbm;
}

}  // namespace

cudaError_t launch_linear_q8(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                             const uint8_t* ws, int64_t N, int64_t K, const void* resid, void* out,
                             bool out_bf16, cudaStream_t st) {
  LinQ8Params p{};
  p.M = M; p.N = N;
  p.kblk = static_cast<int>((K + kKB - 1) / kKB);
  p.xs = xs; p.ws = ws; p.resid = resid; p.out = out;
  p.words = p.kblk % kSG == 0 && reinterpret_cast<uintptr_t>(xs) % 4 == 0 &&
            reinterpret_cast<uintptr_t>(ws) % 4 == 0;
  p.err = device_error_ptr();
  const SkSched sk = sk_sched(M, N, K);
  const bool rows = rows_us(sk, p.kblk) <= pair_us(M, N, p.kblk);
  if (rows)
    return out_bf16 ? launch_rows<__nv_bfloat16>(xq, M, wq, N, K, p, sk, st)
                    : launch_rows<float>(xq, M, wq, N, K, p, sk, st);
  const bool wide = N * (out_bf16 ? 2 : 4) % 32 == 0 && reinterpret_cast<uintptr_t>(out) % 32 == 0 &&
                    reinterpret_cast<uintptr_t>(resid) % 32 == 0;
  if (out_bf16)
    return wide ? launch_pair<__nv_bfloat16, 224, true>(xq, M, wq, N, K, p, st)
                : launch_pair<__nv_bfloat16, 224, false>(xq, M, wq, N, K, p, st);
  return wide ? launch_pair<float, 224, true>(xq, M, wq, N, K, p, st)
              : launch_pair<float, 224, false>(xq, M, wq, N, K, p, st);
}

}  // namespace q3vl
