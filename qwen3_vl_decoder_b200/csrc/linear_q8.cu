// Product of 8-bit rows and an 8-bit weight with block scales (q8.cuh):
//   out[m][n] = sum_j 2^(xs[m][j] + ws[n / 128][j] - 254) sum_{k in block j} xq[m][k] wq[n][k]
// (+ resid[m][n]), summed in fp32 and rounded once.
//
// The tensor core multiplies e4m3 at twice the bf16 rate and, because the
// scales are powers of two, applies them itself (tcgen05.mma kind::mxf8f6f4,
// one scale byte per operand row and 32 columns, here the same byte for the
// four steps of a 128-column block). The partial sums of one output therefore
// stay in one fp32 accumulator over the whole of K, and splitting K needs no
// more than an addition. A warp builds the scale words of each k-block in the
// layout the tensor core reads (q8.cuh), next to the operand tiles that TMA
// brings (128-byte swizzle, 128 columns a box); the MMA thread copies them to
// TMEM in front of the block's four MMAs.
#include "q3vl_internal.h"
#include "q8.cuh"

namespace q3vl {
namespace {

constexpr int kKB = 128;                // k-block: bytes of K per stage and scale
constexpr int kScaleBytes = 512;        // scale words of 128 rows

struct LinQ8Params {
  int64_t M, N;
  int kblk;                // k-blocks: ceil(K / 128)
  const uint8_t* xs;       // [M][kblk]
  const uint8_t* ws;       // [ceil(N / 128)][kblk]
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
  *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void put4(float* o, const float (&v)[4]) {
  *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
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

// ---------------------------------------------------------------------------
// Few rows: the weight is the MMA's M operand (128 rows a tile) and a tile of
// NB <= 224 rows of x its N operand, so that one decoded token pads N to 16
// and not M to 128. Bound by the weight's bytes; K is split over up to 8 CTAs
// of a cluster (about two CTAs per SM stream weights), which leave their fp32
// partial tiles in shared memory and share out the rows of x to add them up
// over DSMEM in split order: the sum has one order whatever the timing.
// ---------------------------------------------------------------------------
constexpr int kSkThreads = 192;         // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue, 2 scales first
constexpr int kSkMaxSplits = 8;         // portable cluster size
constexpr int kSkMaxNB = 224;           // with the scale words 248 TMEM columns: two CTAs per SM

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
  const int sfb = (sc.NB + 127) / 128;                            // scale copies of the x tile
  uint8_t* smA = smem;
  uint8_t* smB = smA + size_t(S) * kABytes;
  uint8_t* smS = smB + size_t(S) * b_bytes;                       // [S][1 + sfb][512]
  uint64_t* full = reinterpret_cast<uint64_t*>(smS + size_t(S) * (1 + sfb) * kScaleBytes);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
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
    // full: the TMA thread and the scale warp; its loads count as bytes
    for (int s = 0; s < S; ++s) { mbar_init(full + s, 2); mbar_init(empty + s, 1); }
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
    if (lane == 0) {
      const int32_t row0 = tile * 128;
      const int pre = n < S ? n : S;
      // the weights may be asked for ahead of the dependency, as far as L2
      for (int i = 0; i < pre; ++i) tma_prefetch_2d(&tmW, (k_lo + i) * kKB, row0);
      griddep_wait();
      int issued = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i % S;
        if (i >= S && !mbar_wait(empty + s, ((i / S) - 1) & 1, p.err, kWhereLinearQ8, abort_flag))
          break;
        mbar_arrive_expect_tx(full + s, kABytes + b_bytes);
        tma_load_2d(smA + size_t(s) * kABytes, &tmW, full + s, (k_lo + i) * kKB, row0);
        tma_load_2d(smB + size_t(s) * b_bytes, &tmX, full + s, (k_lo + i) * kKB,
                    static_cast<int32_t>(m0));
        issued = i + 1;
      }
      // every issued load lands before the CTA may exit
      for (int i = issued - S > 0 ? issued - S : 0; i < issued; ++i)
        mbar_wait(full + (i % S), (i / S) & 1, p.err, kWhereLinearQ8, nullptr);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_mxf8(128, sc.NB);
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int s = i % S;
        if (!mbar_wait(full + s, (i / S) & 1, p.err, kWhereLinearQ8, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // two sets of scale columns in turn, behind the accumulator
        const uint32_t sfa = tmem_base + sc.NB + (i & 1) * 4 * (1 + sfb), sfx = sfa + 4;
        const uint32_t sw = smem_u32(smS + size_t(s) * (1 + sfb) * kScaleBytes);
        tmem_cp_scales(sfa, sdesc_scales(sw));
        for (int c = 0; c < sfb; ++c)
          tmem_cp_scales(sfx + 4 * c, sdesc_scales(sw + (1 + c) * kScaleBytes));
        const uint32_t a0 = smem_u32(smA + size_t(s) * kABytes);
        const uint32_t b0 = smem_u32(smB + size_t(s) * b_bytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_mxf8_ss(tmem_base, sdesc_sw128(a0 + kk * 32, 16, 1024),
                       sdesc_sw128(b0 + kk * 32, 16, 1024), idesc, sfa, sfx,
                       (i | kk) != 0 ? 1u : 0u);
        umma_commit(empty + s);
      }
      if (ok) umma_commit(acc_full);
      else *abort_flag = 1;
    }
    __syncwarp();
  } else {
    griddep_wait();
    if (warp == 2) {
      // scale words of every k-block: one byte for the weight tile, one per
      // row of x (rows past M are zero: any scale)
      uint32_t nx[7], nw;
      auto load = [&](int i) {
        nw = p.ws[int64_t(tile) * p.kblk + k_lo + i];
#pragma unroll
        for (int j = 0; j < 7; ++j) {
          const int r = lane + 32 * j;
          nx[j] = r < sc.NB && m0 + r < p.M ? p.xs[(m0 + r) * p.kblk + k_lo + i] : 127u;
        }
      };
      if (n > 0) load(0);
      for (int i = 0; i < n; ++i) {
        const int s = i % S;
        bool ok = true;
        if (i >= S) {
          if (lane == 0)
            ok = mbar_wait(empty + s, ((i / S) - 1) & 1, p.err, kWhereLinearQ8, abort_flag);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        if (!ok) break;
        uint8_t* w = smS + size_t(s) * (1 + sfb) * kScaleBytes + lane * 16;
        const uint32_t a = nw * 0x01010101u;
        *reinterpret_cast<uint4*>(w) = make_uint4(a, a, a, a);
        *reinterpret_cast<uint4*>(w + kScaleBytes) =
            make_uint4(nx[0] * 0x01010101u, nx[1] * 0x01010101u, nx[2] * 0x01010101u,
                       nx[3] * 0x01010101u);
        if (sfb > 1)
          *reinterpret_cast<uint4*>(w + 2 * kScaleBytes) =
              make_uint4(nx[4] * 0x01010101u, nx[5] * 0x01010101u, nx[6] * 0x01010101u,
                         127u * 0x01010101u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + s);
        if (i + 1 < n) load(i + 1);
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
  __syncthreads();  // all roles done: loads landed, MMAs committed or abandoned
  const bool run = *abort_flag == 0;
  tc_fence_after();
  float* red = reinterpret_cast<float*>(smem);
  const size_t ring = size_t(S) * (kABytes + b_bytes);
  const int rows = static_cast<int>(p.M - m0 < sc.NB ? p.M - m0 : sc.NB);
  int chunk = static_cast<int>(ring / 512) / 16 * 16;  // rows per round
  if (chunk > sc.NB) chunk = sc.NB;
#pragma unroll 1
  for (int j0 = 0; j0 < rows; j0 += chunk) {
    const int nj = rows - j0 < chunk ? rows - j0 : chunk;
    if (warp >= 2 && run) {
      const int q = warp & 3;
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < nj; c0 += 16) {
        uint32_t u[16];
        tmem_ld16(tb + j0 + c0, u);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c0 + c < nj) red[(c0 + c) * 128 + 32 * q + lane] = __uint_as_float(u[c]);
      }
    }
    cluster_sync();  // every CTA's partials of this round are in its shared memory
    if (warp >= 2 && run) {
#pragma unroll 1
      for (int jj = split + (warp - 2) * sc.splits; jj < nj; jj += 4 * sc.splits) {
        const uint32_t own = smem_u32(red + jj * 128 + 4 * lane);
        // every split's values requested before any is added: one DSMEM round
        // trip, then the sum in split order
        float w[kSkMaxSplits][4];
#pragma unroll
        for (int sp = 0; sp < kSkMaxSplits; ++sp) {
          const uint32_t ra = map_to_cta(own, static_cast<uint32_t>(sp < sc.splits ? sp : 0));
#pragma unroll
          for (int i = 0; i < 4; ++i) w[sp][i] = sp < sc.splits ? ld_dsmem_f32(ra + 4u * i) : 0.f;
        }
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int sp = 0; sp < kSkMaxSplits; ++sp)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += w[sp][i];
        finish4<T>(p, m0 + j0 + jj, int64_t(tile) * 128 + 4 * lane, v);
      }
    }
    cluster_sync();  // no CTA overwrites or leaves its buffer while another may read it
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, sc.tcols);
  }
}

SkSched sk_sched(int64_t M, int64_t N, int64_t K) {
  SkSched s;
  s.ttiles = static_cast<int>((M + kSkMaxNB - 1) / kSkMaxNB);
  s.NB = static_cast<int>(((M + s.ttiles - 1) / s.ttiles + 15) / 16 * 16);
  s.tiles = static_cast<int>((N + 127) / 128);
  const int kblk = static_cast<int>((K + kKB - 1) / kKB);
  const int sfb = (s.NB + 127) / 128;
  const size_t stage = size_t(128) * kKB + size_t(s.NB) * kKB + size_t(1 + sfb) * kScaleBytes;
  int st = static_cast<int>(size_t(110 * 1024) / stage);  // two CTAs share an SM
  s.stages = st < 2 ? 2 : (st > 6 ? 6 : st);
  if (s.stages > kblk) s.stages = kblk < 2 ? 2 : kblk;
  s.smem = 1024 + size_t(s.stages) * stage + size_t(2 * s.stages + 1) * 8 + 16;
  while (s.tcols < static_cast<uint32_t>(s.NB + 8 * (1 + sfb))) s.tcols <<= 1;
  const int64_t work = int64_t(s.tiles) * s.ttiles;
  int64_t splits = 2 * int64_t(sm_count()) / work;
  if (splits > kSkMaxSplits) splits = kSkMaxSplits;
  if (splits > kblk) splits = kblk;
  // every tile's cluster inside one GPC (16 SMs counted of each) in the first wave
  const int gpcs = sm_count() / 18 > 1 ? sm_count() / 18 : 1;
  while (splits > 1 && (32 / splits) * gpcs < work) --splits;
  s.splits = static_cast<int>(splits < 1 ? 1 : splits);
  return s;
}

template <typename T>
cudaError_t launch_rows(const uint8_t* xq, int64_t M, const uint8_t* wq, int64_t N, int64_t K,
                        const LinQ8Params& p, cudaStream_t st) {
  const SkSched s = sk_sched(M, N, K);
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

}  // namespace

cudaError_t launch_linear_q8(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                             const uint8_t* ws, int64_t N, int64_t K, const void* resid, void* out,
                             bool out_bf16, cudaStream_t st) {
  LinQ8Params p{};
  p.M = M; p.N = N;
  p.kblk = static_cast<int>((K + kKB - 1) / kKB);
  p.xs = xs; p.ws = ws; p.resid = resid; p.out = out;
  p.err = device_error_ptr();
  if (out_bf16) return launch_rows<__nv_bfloat16>(xq, M, wq, N, K, p, st);
  return launch_rows<float>(xq, M, wq, N, K, p, st);
}

}  // namespace q3vl
