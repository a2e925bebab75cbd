// Making 8-bit blocks (q8.cuh): activation rows behind a residual add and
// RMSNorm, weight matrices, and K/V rows into the 8-bit cache.
#include "q3vl_internal.h"
#include "q8.cuh"

namespace q3vl {
namespace {

// Eight elements of a row as loaded.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    load8(reinterpret_cast<const T*>(v), f);
  }
  // bf16 only: += o, rounded to bf16
  __device__ __forceinline__ void add(const Raw8& o) {
    __nv_bfloat162* a = reinterpret_cast<__nv_bfloat162*>(v);
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(o.v);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = __hadd2(a[j], b[j]);
  }
  // the same as four pairs for the packed arithmetic
  __device__ __forceinline__ void pairs(uint64_t (&f)[4]) const {
    float s[8];
    floats(s);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2_pack(s[2 * j], s[2 * j + 1]);
  }
};

// 1 / sqrt(ss / width + eps) in two parts, ss the sum of the lanes' values (one
// warp). The last two levels of the sum, the quotient and the root keep their
// remainders, to 2^-40 of the result; what is left is half the error of the sum
// before: up to 13 roundings of 2^-24 (four squares and sums, the two halves of
// a pair, five levels in a warp, three here), 25 in rows wider than 8192.
__device__ __forceinline__ float2 inv_rms(float ss, float width, float eps) {
#pragma unroll
  for (int o = 16; o > 2; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  float lo = 0.f;
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, ss, o), yl = __shfl_xor_sync(0xffffffffu, lo, o);
    const float z = ss + y, b = z - ss;
    lo = (lo + yl) + ((ss - (z - b)) + (y - b));
    ss = z;
  }
  const float q = ss / width;
  const float ql = (fmaf(-q, width, ss) + lo) / width;
  const float var = q + eps, b = var - q;
  const float vl = ql + ((q - (var - b)) + (eps - b));
  const float inv = 1.0f / sqrtf(var);
  // (var + vl) inv^2 = 1 - d, so 1 / sqrt(var + vl) = inv (1 + d / 2)
  const float a = var * inv, al = fmaf(var, inv, -a);
  float il = 0.5f * inv * (fmaf(-a, inv, 1.f) - (al + vl * inv) * inv);
  if (!(fabsf(il) < inv)) il = 0.f;  // var 0 or not finite
  return make_float2(inv, il);
}

// Whether a bf16 gain is one of those (finite, 2^64 and more) whose product with
// an element may leave fp32 where h / rms * gain does not; elements are below
// 2^64 while the sum of squares is finite. They are refused: a power of two of
// 1 / rms put in front of the product would take them in, for 3 to 7% of the time.
__device__ __forceinline__ bool far_gain(const Raw8<__nv_bfloat16>& g) {
  float v[8];
  g.floats(v);
  bool far = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) far |= fabsf(v[j]) >= 0x1p64f && fabsf(v[j]) < INFINITY;
  return far;
}
__device__ __forceinline__ bool far_gain(const Raw8<float>&) { return false; }  // h / rms first

// v = h / rms * gain / scale was rounded onto the middle of two e4m3 steps:
// the neighbour on the side on which h * gain * (inv + inv_lo) lies (one value
// in a million; below 2^-6, where e4m3 has fewer bits, a middle keeps its
// rounding). Right where the row's sum is: rows with exact sums get the bytes of
// 64-bit arithmetic, of others see below.
__device__ __noinline__ float off_middle(float v, float h, float gain, float inv, float inv_lo,
                                         float s) {
  const double y = fabs(double(h) * double(gain) * (double(inv) + double(inv_lo)) * double(s));
  const double m = fabs(double(v));
  const uint32_t bits = __float_as_uint(v);
  return __uint_as_float(y > m ? bits + 1 : y < m ? bits - 1 : bits);
}

// ---------------------------------------------------------------------------
// h = x + delta; y = h * (1 / rms(h)) * gain; e4m3 of y, a scale per 128
// columns. A block takes rows blockIdx.x, + gridDim.x, ...; a thread takes
// units of 8 columns, so 16 neighbouring threads hold one block of 128 and its
// maximum is four shuffles. The row stays in registers between the sum of
// squares (fp32) and the rounding: every input is read once. Bound by memory:
// 7 bytes per bf16 element with a delta (3 without). Rows up to 8192 wide (NV =
// 1) go through as many blocks as fit, which request the next row before they
// reduce this one; that wants 48 registers, for three quarters of the threads.
// Instructions come close behind memory, hence the packed arithmetic and the
// branches for what only infinities need. One warp makes 1 / rms for the block.
// Measured: bf16 with a delta 4096 x 2560 15.1 us, 8192 x 5120 55.7 (5.3 TB/s),
// fp32 2129 x 5120 15.3; with an fp32 1 / rms made by every warp 14.7, 52, 14.4.
// Before that step a block per row without look-ahead took 18.2, 75, 19.3, and a
// ring of bulk copies instead of registers 18.9 at the first size. Of 67 million
// random values 4 to 22 in rows of up to 5120, and 0 to 9 in wider ones, got
// another e4m3 value than from 64-bit arithmetic, 31 to 64 by fp32 operations
// one after the other. The scale is that of the fp32 values: a maximum that
// rounds onto 448 scales keeps the smaller one.
// ---------------------------------------------------------------------------
template <typename T, int NV, bool PRE, bool DELTA>
__global__ void __maxnreg__(NV == 1 ? 48 : 64)
add_rms_norm_q8_kernel(const T* x, const T* delta, const T* gain, T* h, uint8_t* q,
                       uint8_t* scales, int64_t rows, int width, int nblk, float eps,
                       int32_t* err) {
  const int t = threadIdx.x, lane = t & 31;
  const int units = width / 8;
  __shared__ float s_ss[2][32];
  __shared__ float2 s_inv[2];
  griddep_launch_dependents();
  griddep_wait();
  Raw8<T> xn, dn, gn;
  auto request = [&](int64_t row, int u) {
    xn.zero();
    dn.zero();
    if (u < units) {
      xn.load(x + row * width + 8 * u);
      if (DELTA) dn.load(delta + row * width + 8 * u);
    }
  };
  auto request_gain = [&](int u) {
    gn.zero();
    if (gain != nullptr && u < units) gn.load(gain + 8 * u);
  };
  if (PRE) request(blockIdx.x, t);
  if (NV == 1) request_gain(t);
  if (sizeof(T) == 2 && blockIdx.x == 0) {
    for (int u = t; u < NV * int(blockDim.x); u += blockDim.x) {
      if (NV > 1) request_gain(u);
      if (far_gain(gn)) record_error(err, Q3VL_ERANGE, kWhereNormQ8Gain);
    }
  }
  int par = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, par ^= 1) {
    uint64_t f[NV][4];  // two elements each: packed fp32 arithmetic
    uint64_t ss2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = t + i * blockDim.x;
      if (!PRE) request(row, u);
      if constexpr (DELTA && sizeof(T) == 2) {
        // A sum of two bf16 that is inexact in fp32 has one of them below 2^-16
        // of the other, and rounds to that other either way: so a packed bf16
        // addition gives the bits of the fp32 sum rounded to bf16.
        xn.add(dn);
        if (u < units) *reinterpret_cast<uint4*>(h + row * width + 8 * u) = xn.v[0];
      }
      xn.pairs(f[i]);
      if constexpr (DELTA && sizeof(T) == 4) {
        uint64_t d[4];
        dn.pairs(d);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f2_unpack(f2_add(f[i][j], d[j]), v[2 * j], v[2 * j + 1]);
        if (u < units) store8(h + row * width + 8 * u, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i][j] = f2_pack(v[2 * j], v[2 * j + 1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) ss2 = f2_fma(f[i][j], f[i][j], ss2);
    }
    if (PRE && row + gridDim.x < rows) request(row + gridDim.x, t);
    float inv = 1.f, inv_lo = 0.f;  // 1 / rms in two parts
    if (gain != nullptr) {
      float ss, ss1;
      f2_unpack(ss2, ss, ss1);
      ss = warp_sum(ss + ss1);
      if (lane == 0) s_ss[par][t >> 5] = ss;
      __syncthreads();
      if (t < 32) {
        const float2 r = inv_rms(lane < (blockDim.x >> 5) ? s_ss[par][lane] : 0.f,
                                 static_cast<float>(width), eps);
        if (lane == 0) s_inv[par] = r;
      }
      __syncthreads();
      inv = s_inv[par].x;
      inv_lo = s_inv[par].y;
    }
    const uint64_t inv2 = f2_pack(inv, inv), minus2 = f2_pack(-inv, -inv),
                   lo2 = f2_pack(inv_lo, inv_lo);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = t + i * blockDim.x;
      if (NV > 1) request_gain(u);
      if (gain != nullptr) {
        uint64_t g[4];
        gn.pairs(g);
        if (sizeof(T) == 2 && inv == 0.f) {  // the sum overflowed: zeros, whatever the gain
#pragma unroll
          for (int j = 0; j < 4; ++j) f[i][j] = f2_mul(f[i][j], 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // f * inv * g rounded once: about one value in a million lies so
          // near a border of e4m3 that an error in the last place turns it
          // over, and rounding f * inv as well turned over two to three times
          // as many. What lands on a border all the same goes to off_middle.
          // A product of two bf16 is exact.
          if constexpr (sizeof(T) == 2) {
            const uint64_t fg = f2_mul(f[i][j], g[j]);
            f[i][j] = f2_fma(fg, inv2, f2_mul(fg, lo2));
          } else {
            const uint64_t y = f2_mul(f[i][j], inv2);
            const uint64_t rest =
                f2_fma(f[i][j], lo2, f2_fma(f[i][j], inv2, f2_mul(f[i][j], minus2)));
            f[i][j] = f2_fma(y, g[j], f2_mul(rest, g[j]));
          }
        }
      }
      float v[8], a = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f2_unpack(f[i][j], v[2 * j], v[2 * j + 1]);
        a = fmaxf(a, fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));  // leaves NaN out
      }
      const bool infinite = __any_sync(0xffffffffu, a == INFINITY);
      if (infinite) {
        a = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_abs(v[j]));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const uint32_t e = e8m0_of_amax(a);
      const float s = e8m0_inverse(e);
      const uint64_t s2 = f2_pack(s, s);
#pragma unroll
      for (int j = 0; j < 4; ++j) f2_unpack(f2_mul(f[i][j], s2), v[2 * j], v[2 * j + 1]);
      if (infinite) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], 0.f, v[j]);
      }
      if (gain != nullptr) {
        // low 20 bits 0x80000: rounded onto the middle of two steps
        uint32_t low = ~0u;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          low = min(low, __float_as_uint(v[j]) * 4096u + 0x80000000u);
        if (low == 0 && u < units) {
          const T* hr = (DELTA ? h : x) + row * width + 8 * u;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if ((__float_as_uint(v[j]) & 0xfffffu) == 0x80000u)
              v[j] = off_middle(v[j], static_cast<float>(hr[j]),
                                static_cast<float>(gain[8 * u + j]), inv, inv_lo, s);
        }
      }
      if (u < units) {
        uint2 w;
        w.x = pack_e4m3x4_finite(v[0], v[1], v[2], v[3]);
        w.y = pack_e4m3x4_finite(v[4], v[5], v[6], v[7]);
        *reinterpret_cast<uint2*>(q + row * width + 8 * u) = w;
        if ((t & 15) == 0) scales[row * nblk + u / 16] = static_cast<uint8_t>(e);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Weights: one block of 256 threads per 128 x 128 block, whose elements stay
// in registers between the maximum and the rounding.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
quantize_weight_kernel(const T* __restrict__ w, int64_t N, int64_t K, uint8_t* __restrict__ wq,
                       uint8_t* __restrict__ ws) {
  const int t = threadIdx.x, lane = t & 31;
  const int64_t kblk = (K + 127) / 128;
  const int64_t nb = blockIdx.x / kblk, kb = blockIdx.x % kblk;
  const int64_t col = kb * 128 + (t & 15) * 8;
  float f[8][8];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = nb * 128 + (t >> 4) + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    if (row < N && col < K) load8(w + row * K + col, f[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_abs(f[i][j]));
  }
  __shared__ float s_a[8];
  a = warp_max(a);
  if (lane == 0) s_a[t >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, s_a[i]);
  const uint32_t e = e8m0_of_amax(a);
  const float s = e8m0_inverse(e);
  if (t == 0) ws[nb * kblk + kb] = static_cast<uint8_t>(e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = nb * 128 + (t >> 4) + 16 * i;
    if (row < N && col < K) {
      uint2 v;
      v.x = pack_e4m3x4(f[i][0] * s, f[i][1] * s, f[i][2] * s, f[i][3] * s);
      v.y = pack_e4m3x4(f[i][4] * s, f[i][5] * s, f[i][6] * s, f[i][7] * s);
      *reinterpret_cast<uint2*>(wq + row * K + col) = v;
    }
  }
}

// ---------------------------------------------------------------------------
// Rows into the 8-bit cache. A work item is one (sequence, 128-token block,
// KV head, K or V); its new rows stay in registers between the maximum and
// the rounding. The items of sequence b sit at floor(starts[b] / 128) + 2 b
// along grid x: n rows touch at most floor(n / 128) + 2 blocks, so the items
// of two sequences never meet and no scan is needed; a place that no item
// takes exits. Bound by memory, 3 bytes per element, and by instructions: the
// maximum is taken on pairs of bf16 as they were loaded and infinities are left
// to a branch (15000 rows of 8 heads, K and V, 19.0 us or 4.9 TB/s; 22.2 with
// the finite magnitudes picked out one by one).
// ---------------------------------------------------------------------------
struct StoreQ8Params {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t ld, T;
  const int32_t* starts;  // [B + 1] or null: one row per sequence (seq given), or all T rows
  int B;
  const int32_t* seq;     // [B] or null: slot seq0, from row 0
  const int32_t* len;     // [B]
  int32_t seq0;
  uint8_t* kc;
  uint8_t* vc;
  uint8_t* ks;
  uint8_t* vs;
  int64_t cap;
  int n_seq, nkv;
  int32_t* err;
};

__global__ void __launch_bounds__(256, 4) kv_store_q8_kernel(StoreQ8Params p) {
  const int t = threadIdx.x, lane = t & 31;
  __shared__ int s_item[4];  // slot (-1: none), rows cached, first source row, rows
  __shared__ int s_blk;
  __shared__ float s_a[2][8];
  if (t == 0) s_item[0] = -1;
  griddep_launch_dependents();
  griddep_wait();
  __syncthreads();
  // Starts that decrease would let two sequences claim one place: then nothing
  // is stored. B <= 256: one sequence per thread.
  bool falls = false;
  if (t < p.B) {
    const int b = t;
    int slot, len, s0;
    int64_t rows;  // of two starts of any value
    if (p.seq == nullptr) {
      slot = p.seq0; len = 0; s0 = 0; rows = p.T;
    } else {
      slot = p.seq[b];
      len = p.len[b];
      s0 = p.starts ? p.starts[b] : b;
      rows = int64_t(p.starts ? p.starts[b + 1] : b + 1) - s0;
    }
    falls = rows < 0;
    const bool ok = slot >= 0 && slot < p.n_seq && len >= 0 && rows >= 0 && s0 >= 0 &&
                    s0 + rows <= p.T && len + rows <= p.cap;
    const int n = ok ? static_cast<int>(rows) : 0;
    if (!ok && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
      record_error(p.err, Q3VL_ERANGE, kWhereStoreQ8Range);
    const int64_t base = p.starts ? int64_t(s0) / 128 + 2 * b : b;
    const int64_t j = int64_t(blockIdx.x) - base;
    if (ok && n > 0 && j >= 0 && j <= (len + n - 1) / 128 - len / 128) {
      s_item[0] = slot; s_item[1] = len; s_item[2] = s0; s_item[3] = n;
      s_blk = len / 128 + static_cast<int>(j);
    }
  }
  if (__syncthreads_or(falls ? 1 : 0)) return;
  const int slot = s_item[0];
  if (slot < 0) return;
  const int len = s_item[1], n = s_item[3], blk = s_blk;
  const int g = blockIdx.y;
  const __nv_bfloat16* src = (blockIdx.z == 0 ? p.k : p.v) + int64_t(g) * 128 + (t & 15) * 8;
  uint8_t* cache = blockIdx.z == 0 ? p.kc : p.vc;
  const int64_t nblk = (p.cap + 127) / 128;
  uint8_t* scale = (blockIdx.z == 0 ? p.ks : p.vs) + (int64_t(slot) * nblk + blk) * p.nkv + g;
  const int lo = max(len, blk * 128), hi = min(len + n, blk * 128 + 128);
  const int64_t s0 = int64_t(s_item[2]) + (lo - len);
  Raw8<__nv_bfloat16> f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = (t >> 4) + 16 * i;
    f[i].zero();
    if (lo + r < hi && dcheck(s0 + r < p.T, p.err, kWhereDbgQ8)) f[i].load(src + (s0 + r) * p.ld);
  }
  // The largest magnitude, two elements to a word; NaN drops out. An infinity
  // is rare enough for a second look at the block, that leaves it out.
  auto block_max = [&](float v, int set) {
    v = warp_max(v);
    if (lane == 0) s_a[set][t >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) v = fmaxf(v, s_a[set][i]);
    return v;
  };
  __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {f[i].v[0].x, f[i].v[0].y, f[i].v[0].z, f[i].v[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[j])));
  }
  const bool keeps = blk * 128 < len;  // the block holds earlier rows
  const uint32_t was = keeps ? *scale : 0u;
  float a = block_max(fmaxf(__low2float(top), __high2float(top)), 0);
  const bool infinite = a == INFINITY;
  if (infinite) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      f[i].floats(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_abs(v[j]));
    }
    a = block_max(a, 1);
  }
  uint32_t e = e8m0_of_amax(a);
  if (keeps && was >= e) e = was;
  if (t == 0) *scale = static_cast<uint8_t>(e);
  const int64_t rs = int64_t(p.nkv) * 128;
  uint8_t* dst = cache + (int64_t(slot) * p.cap) * rs + int64_t(g) * 128 + (t & 15) * 8;
  if (keeps && e > was) {
    // the earlier rows move to the larger scale: a shift of the exponent, and
    // a rounding of what falls among e4m3's subnormals
    const float m = e - was > 126 ? 0.f : e8m0_inverse(127 + (e - was));
    for (int r = blk * 128 + (t >> 4); r < len; r += 16) {
      uint2 w = *reinterpret_cast<uint2*>(dst + r * rs);
      const float4 x = unpack_e4m3x4(w.x), y = unpack_e4m3x4(w.y);
      w.x = pack_e4m3x4(x.x * m, x.y * m, x.z * m, x.w * m);
      w.y = pack_e4m3x4(y.x * m, y.y * m, y.z * m, y.w * m);
      *reinterpret_cast<uint2*>(dst + r * rs) = w;
    }
  }
  const float s = e8m0_inverse(e);
  const uint64_t s2 = f2_pack(s, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = lo + (t >> 4) + 16 * i;
    if (r < hi && dcheck(r < p.cap, p.err, kWhereDbgQ8)) {
      uint64_t x[4];
      float v[8];
      f[i].pairs(x);
#pragma unroll
      for (int j = 0; j < 4; ++j) f2_unpack(f2_mul(x[j], s2), v[2 * j], v[2 * j + 1]);
      if (infinite) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], 0.f, v[j]);
      }
      uint2 w;
      w.x = pack_e4m3x4_finite(v[0], v[1], v[2], v[3]);
      w.y = pack_e4m3x4_finite(v[4], v[5], v[6], v[7]);
      *reinterpret_cast<uint2*>(dst + int64_t(r) * rs) = w;
    }
  }
}

__global__ void iota_zero_kernel(int B, int32_t* iota, int32_t* zero) {
  const int b = threadIdx.x;
  if (b >= B) return;
  iota[b] = b;
  zero[b] = 0;
}

template <typename T>
cudaError_t launch_norm_t(const void* x, const void* delta, int64_t S, const void* gain, void* h,
                          uint8_t* q, uint8_t* scales, int width, float eps, cudaStream_t st) {
  const int units = width / 8;
  const int nblk = (width + kQ8Block - 1) / kQ8Block;
  auto go = [&](auto kern, int nv, bool pre) {
    const int th = ((units + nv - 1) / nv + 31) / 32 * 32;
    int64_t blocks = S;
    if (pre) {
      int n = 0;
      const cudaError_t e = max_active_blocks(reinterpret_cast<const void*>(kern), th, &n);
      if (e != cudaSuccess) return e;
      const int64_t fit = int64_t(sm_count()) * (n > 0 ? n : 1);
      if (blocks > fit) blocks = fit;
    }
    return launch_pdl_plain(kern, dim3(static_cast<unsigned>(blocks)), dim3(th), 0, st,
                            static_cast<const T*>(x), static_cast<const T*>(delta),
                            static_cast<const T*>(gain), static_cast<T*>(h), q, scales, S, width,
                            nblk, eps, device_error_ptr());
  };
  cudaError_t e;
  if (units <= 1024)
    e = delta != nullptr ? go(add_rms_norm_q8_kernel<T, 1, true, true>, 1, true)
                         : go(add_rms_norm_q8_kernel<T, 1, true, false>, 1, true);
  else if (units <= 4096)
    e = delta != nullptr ? go(add_rms_norm_q8_kernel<T, 4, false, true>, 4, false)
                         : go(add_rms_norm_q8_kernel<T, 4, false, false>, 4, false);
  else
    return cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  return counted_launch(1);
}

}  // namespace

cudaError_t launch_add_rms_norm_q8(const q3vl_config& c, const void* x, const void* delta, int64_t S,
                                   const void* gain, void* h, uint8_t* q, uint8_t* scales,
                                   cudaStream_t st) {
  const float eps = static_cast<float>(c.rms_eps);
  if (c.dtype == Q3VL_DTYPE_BF16)
    return launch_norm_t<__nv_bfloat16>(x, delta, S, gain, h, q, scales, c.hidden, eps, st);
  return launch_norm_t<float>(x, delta, S, gain, h, q, scales, c.hidden, eps, st);
}

cudaError_t launch_quantize_weight_q8(const q3vl_config& c, const void* w, int64_t N, int64_t K,
                                      uint8_t* wq, uint8_t* ws, cudaStream_t st) {
  const int64_t blocks = ((N + 127) / 128) * ((K + 127) / 128);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (c.dtype == Q3VL_DTYPE_BF16)
    quantize_weight_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(
        static_cast<const __nv_bfloat16*>(w), N, K, wq, ws);
  else
    quantize_weight_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(
        static_cast<const float*>(w), N, K, wq, ws);
  return counted_launch(1);
}

cudaError_t launch_kv_store_q8(const q3vl_config& c, const void* k, const void* v, int64_t ld,
                               int64_t T, const int32_t* starts, int B,
                               const q3vl_kv_cache_q8& kv, const int32_t* seq, const int32_t* len,
                               int32_t seq0, cudaStream_t st) {
  StoreQ8Params p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.ld = ld; p.T = T; p.starts = starts; p.B = B; p.seq = seq; p.len = len; p.seq0 = seq0;
  p.kc = kv.k; p.vc = kv.v; p.ks = kv.k_scale; p.vs = kv.v_scale;
  p.cap = kv.cap; p.n_seq = kv.n_seq; p.nkv = c.n_kv_heads;
  p.err = device_error_ptr();
  // places along x: see the kernel's comment
  const int64_t nx = starts ? T / 128 + 2 * int64_t(B) : (seq ? B : (T + 127) / 128);
  const cudaError_t e = launch_pdl_plain(
      kv_store_q8_kernel,
      dim3(static_cast<unsigned>(nx), static_cast<unsigned>(c.n_kv_heads), 2), dim3(256), 0, st, p);
  if (e != cudaSuccess) return e;
  return counted_launch(1);
}

cudaError_t launch_iota_zero(int B, int32_t* iota, int32_t* zero, cudaStream_t st) {
  iota_zero_kernel<<<1, 256, 0, st>>>(B, iota, zero);
  return counted_launch(1);
}

}  // namespace q3vl
