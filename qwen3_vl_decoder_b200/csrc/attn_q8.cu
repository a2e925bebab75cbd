// Attention of one query row per sequence over the 8-bit cache (q8.cuh).
#include "q3vl_internal.h"
#include "q8.cuh"

namespace q3vl {
namespace {

struct AttnQ8Params {
  const __nv_bfloat16* q;   // [B][nh*128]
  const uint8_t* kc;        // the cache [n_seq][cap][nkv*128]
  const uint8_t* vc;
  const uint8_t* ks;        // scales [n_seq][nblk][nkv]
  const uint8_t* vs;
  int64_t cap;
  int n_seq, nblk;
  const int32_t* seq;
  const int32_t* len;
  int plus;
  int B, nkv, G;
  float scale_log2;         // log2(e) / sqrt(128)
  __nv_bfloat16* o;         // [B][nh*128]
  int32_t* err;
};

// One block of 128 threads per (sequence, query head): thread t scores token
// t of each 128-token block, then sums dimension t over the block's tokens.
__global__ void __launch_bounds__(128) attn_q8_kernel(AttnQ8Params p) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int nh = p.G * p.nkv, b = blockIdx.x / nh, h = blockIdx.x % nh, g = h / p.G;
  __shared__ float s_q[128], s_p[128], s_r[4];
  griddep_wait();
  const int slot = p.seq[b], L = p.len[b] + p.plus;
  const bool ok = slot >= 0 && slot < p.n_seq && L >= p.plus && int64_t(L) <= p.cap;
  if (!ok && t == 0) record_error(p.err, Q3VL_ERANGE, kWhereAttnQ8Range);
  const int n = ok ? L : 0;
  s_q[t] = __bfloat162float(p.q[(int64_t(b) * nh + h) * 128 + t]) * p.scale_log2;
  __syncthreads();
  const int64_t rs = int64_t(p.nkv) * 128;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int c = 0; c * 128 < n; ++c) {
    const int64_t row0 = int64_t(slot) * p.cap + c * 128;
    const int64_t si = (int64_t(slot) * p.nblk + c) * p.nkv + g;
    float s = -INFINITY;
    if (c * 128 + t < n) {
      const uint32_t* kr = reinterpret_cast<const uint32_t*>(p.kc + (row0 + t) * rs + g * 128);
      float d = 0.f;
      for (int i = 0; i < 32; ++i) {
        const float4 x = unpack_e4m3x4(kr[i]);
        d += x.x * s_q[4 * i] + x.y * s_q[4 * i + 1] + x.z * s_q[4 * i + 2] + x.w * s_q[4 * i + 3];
      }
      s = d * e8m0_scale(p.ks[si]);
    }
    float w = warp_max(s);
    if (lane == 0) s_r[warp] = w;
    __syncthreads();
    const float M = fmaxf(m, fmaxf(fmaxf(s_r[0], s_r[1]), fmaxf(s_r[2], s_r[3])));
    const float e = s == -INFINITY ? 0.f : exp2f(s - M);
    s_p[t] = e;
    __syncthreads();
    w = warp_sum(e);
    if (lane == 0) s_r[warp] = w;
    __syncthreads();
    const float a = m == -INFINITY ? 0.f : exp2f(m - M);
    l = l * a + (s_r[0] + s_r[1] + s_r[2] + s_r[3]);
    float o = 0.f;
    for (int i = 0; i < 128 && c * 128 + i < n; ++i) {
      const uint32_t x = p.vc[(row0 + i) * rs + g * 128 + t];
      o += s_p[i] * unpack_e4m3x4(x).x;
    }
    acc = acc * a + o * e8m0_scale(p.vs[si]);
    m = M;
    __syncthreads();
  }
  p.o[(int64_t(b) * nh + h) * 128 + t] = __float2bfloat16_rn(n > 0 ? acc / l : 0.f);
}

}  // namespace

size_t attention_q8_ws_bytes(const q3vl_config& c, int B, int64_t cap) {
  (void)c; (void)B; (void)cap;
  return 256;
}

cudaError_t launch_attention_q8(const q3vl_config& c, const void* q, int B,
                                const q3vl_kv_cache_q8& kv, const int32_t* seq,
                                const int32_t* len, int plus, bool early, void* o, void* ws,
                                cudaStream_t st) {
  (void)early; (void)ws;
  AttnQ8Params p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kc = kv.k; p.vc = kv.v; p.ks = kv.k_scale; p.vs = kv.v_scale;
  p.cap = kv.cap; p.n_seq = kv.n_seq; p.nblk = static_cast<int>((kv.cap + 127) / 128);
  p.seq = seq; p.len = len; p.plus = plus;
  p.B = B; p.nkv = c.n_kv_heads; p.G = c.n_heads / c.n_kv_heads;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / 11.313708498984761);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.err = device_error_ptr();
  const cudaError_t e = launch_pdl_plain(attn_q8_kernel, dim3(B * c.n_heads), dim3(128), 0, st, p);
  if (e != cudaSuccess) return e;
  return counted_launch(1);
}

}  // namespace q3vl
