// Projections with 4-bit weights (moe_linear): y = x W^T + b, W in the
// experts' format (codes with one binary16 scale per 32 inputs).
//
// Batches of up to 32 tokens, in bf16 or in 8 bits with scales: the work is
// reading W once (0.5625 bytes per weight), so the weights go straight from
// HBM into registers and are multiplied there with the legacy tensor path
// (mma.sync): W is the 16-row operand A, unpacked exactly to bf16 integers
// (code - 8), up to four 8-token column tiles are operand B, and the fp32
// result of every 32-input block is multiplied by the block's scale.  No
// weight and no activation is rounded.
#include <math.h>

#include <new>

#include "device_common.cuh"
#include "linear_internal.cuh"
#include "op_common.cuh"
#include "profile.cuh"

namespace moe {
namespace lin {
namespace {

using namespace dev;
using namespace op;

// ------------------------------------------------------------ packing
__global__ void pack_kernel(const uint8_t* __restrict__ q, const uint16_t* __restrict__ s, int N, int K, int kc,
                            uint8_t* __restrict__ tiles) {
  // one warp per tile
  const size_t tile = (size_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const size_t n_tiles = (size_t)((N + kTileRows - 1) / kTileRows) * kc;
  if (tile >= n_tiles) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int row0 = (int)(tile / kc) * kTileRows, k0 = (int)(tile % kc) * kTileK;
  uint8_t* dst = tiles + tile * kTileBytes;
  for (int half = 0; half < 2; ++half) {
    uint32_t w[4];
    for (int i = 0; i < 4; ++i) {
      const int row = row0 + g + 8 * (i & 1), k = k0 + 64 * half + 32 * (i >> 1) + 8 * t;
      uint32_t v = 0x88888888u;  // code 8: weight 0
      if (row < N && k < K) {
        const uint8_t* b = q + (size_t)row * (K / 2) + k / 2;  // four bytes: inputs k .. k + 7
        v = 0;
        for (int j = 0; j < 4; ++j) v |= (uint32_t)(b[j] & 15) << (4 * j) | (uint32_t)(b[j] >> 4) << (4 * j + 16);
      }
      w[i] = v;
    }
    *reinterpret_cast<uint4*>(dst + 512 * half + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  for (int i = lane; i < 64; i += 32) {  // scale i: 8 g' + (0..3 row g', 4..7 row g' + 8)
    const int row = row0 + (i >> 3) + 8 * ((i >> 2) & 1), blk = k0 / 32 + (i & 3);
    reinterpret_cast<uint16_t*>(dst + kTileCodes)[i] =
        (row < N && blk < K / 32) ? s[(size_t)row * (K / 32) + blk] : (uint16_t)0;
  }
}

// ------------------------------------------------------------ small batches
struct SmallParams {
  Weights w;
  const uint16_t* x;   // [T][K] bf16, or
  const int8_t* q;     // [T][K] codes and
  const float* qs;     // [T][K/32] scales
  uint16_t* y;         // [T][N] bf16
  int T;
};

// D += A B, A 16x16 (rows x inputs), B 16x8 (inputs x tokens), bf16 -> fp32
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pair i of a word as bf16 integers code - 8: a 4-bit code ORed into the
// mantissa of 128.0 reads 128 + code, and the difference to 136 is exact.
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int i) {
  const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 k136 = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), k136);
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Four signed bytes as two words of bf16 pairs (exact: |code| <= 128).
__device__ __forceinline__ void bytes_to_bf16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  lo = pack_bf16((float)(int8_t)(c & 0xff), (float)(int8_t)((c >> 8) & 0xff));
  hi = pack_bf16((float)(int8_t)((c >> 16) & 0xff), (float)(int8_t)(c >> 24));
}

// CTAs of 8 warps; S warps share a 16-row tile, each with a contiguous part
// of the K tiles (their partial sums meet in shared memory, in one fixed
// order).  A warp streams its tiles through a ring of kRing register sets.
template <int NT, int S, bool kQ8>
__global__ void __launch_bounds__(256, 2) small_kernel(const __grid_constant__ SmallParams p) {
  constexpr int kRing = 3;
  __shared__ float part[S > 1 ? 8 * 32 * 4 * NT : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kc = p.w.kc, K = p.w.K;
  const int c0 = (warp % S) * kc / S, c1 = (warp % S + 1) * kc / S;
  const int tstep = gridDim.x * (8 / S);
  const int tile0 = blockIdx.x * (8 / S) + warp / S;

  uint4 wa[kRing], wb[kRing], ws[kRing];
  int lt = tile0, lc = c0;  // next tile to load
  auto load = [&](int slot) {
    if (lt < p.w.nt && lc < c1) {
      const uint8_t* src = p.w.tiles + ((size_t)lt * kc + lc) * kTileBytes;
      wa[slot] = ld_stream(src + 16 * lane);
      wb[slot] = ld_stream(src + 512 + 16 * lane);
      ws[slot] = ld_stream(src + kTileCodes + 16 * g);
      if (++lc == c1) lc = c0, lt += tstep;
    }
  };
#pragma unroll
  for (int i = 0; i < kRing; ++i) load(i);  // the weights are the library's own: nothing to wait for
  dep_wait();
  dep_release();

  for (int tile = tile0; tile - warp / S < p.w.nt; tile += tstep) {  // uniform over the CTA
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    if (tile < p.w.nt) {
      for (int cb = c0; cb < c1; ++cb) {
        const uint32_t words[8] = {wa[0].x, wa[0].y, wa[0].z, wa[0].w, wb[0].x, wb[0].y, wb[0].z, wb[0].w};
        const uint4 sc = ws[0];
#pragma unroll
        for (int i = 0; i + 1 < kRing; ++i) wa[i] = wa[i + 1], wb[i] = wb[i + 1], ws[i] = ws[i + 1];
        load(kRing - 1);
        const __half2 sg01 = *reinterpret_cast<const __half2*>(&sc.x), sg23 = *reinterpret_cast<const __half2*>(&sc.y);
        const __half2 sh01 = *reinterpret_cast<const __half2*>(&sc.z), sh23 = *reinterpret_cast<const __half2*>(&sc.w);
        const float sg[4] = {__low2float(sg01), __high2float(sg01), __low2float(sg23), __high2float(sg23)};
        const float sh[4] = {__low2float(sh01), __high2float(sh01), __low2float(sh23), __high2float(sh23)};
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int k = cb * kTileK + 32 * b;
          if (k >= K) break;
          uint32_t a[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[0][i] = unpack_pair(words[2 * b], i);
            a[1][i] = unpack_pair(words[2 * b + 1], i);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int tok = 8 * n + g;
            uint4 xv = make_uint4(0u, 0u, 0u, 0u);
            float f0 = 1.0f, f1 = 1.0f;
            if constexpr (kQ8) {
              if (tok < p.T) {
                const uint2 c = *reinterpret_cast<const uint2*>(p.q + (size_t)tok * K + k + 8 * t);
                bytes_to_bf16(c.x, xv.x, xv.y);
                bytes_to_bf16(c.y, xv.z, xv.w);
              }
              const int t0 = 8 * n + 2 * t;
              f0 = t0 < p.T ? p.qs[(size_t)t0 * (K >> 5) + (k >> 5)] : 0.0f;
              f1 = t0 + 1 < p.T ? p.qs[(size_t)(t0 + 1) * (K >> 5) + (k >> 5)] : 0.0f;
            } else {
              if (tok < p.T) xv = *reinterpret_cast<const uint4*>(p.x + (size_t)tok * K + k + 8 * t);
            }
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_bf16(d, a[0][0], a[1][0], a[0][1], a[1][1], xv.x, xv.y);
            mma_bf16(d, a[0][2], a[1][2], a[0][3], a[1][3], xv.z, xv.w);
            if constexpr (kQ8) {
              d[0] *= f0, d[1] *= f1, d[2] *= f0, d[3] *= f1;
            }
            acc[n][0] = fmaf(sg[b], d[0], acc[n][0]);
            acc[n][1] = fmaf(sg[b], d[1], acc[n][1]);
            acc[n][2] = fmaf(sh[b], d[2], acc[n][2]);
            acc[n][3] = fmaf(sh[b], d[3], acc[n][3]);
          }
        }
      }
    }
    if constexpr (S > 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float4*>(&part[((warp * NT + n) * 32 + lane) * 4]) =
            make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
      __syncthreads();
      if (warp % S == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 1; i < S; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(&part[(((warp + i) * NT + n) * 32 + lane) * 4]);
            acc[n][0] += v.x, acc[n][1] += v.y, acc[n][2] += v.z, acc[n][3] += v.w;
          }
      }
      __syncthreads();
    }
    if (tile < p.w.nt && warp % S == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = tile * kTileRows + g + 8 * h;
        if (row < p.w.N) {
          const float bias = p.w.bias ? __ldg(p.w.bias + row) : 0.0f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int tok = 8 * n + 2 * t + i;
              if (tok < p.T)
                p.y[(size_t)tok * p.w.N + row] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[n][2 * h + i] + bias));
            }
        }
      }
    }
  }
}

template <int NT, bool kQ8>
cudaError_t launch_small_nt(const SmallParams& p, int num_sms, cudaStream_t s) {
  // warps per tile: enough to give every SM 16 warps
  const int want = num_sms * 16;
  int S = 1;
  while (S < 8 && p.w.nt * S < want && 2 * S <= p.w.kc) S *= 2;
  const int per = 8 / S;
  const int grid = min((p.w.nt + per - 1) / per, 2 * num_sms);
  switch (S) {
    case 1: return launch_overlapped(small_kernel<NT, 1, kQ8>, dim3(grid), dim3(256), 0, s, p);
    case 2: return launch_overlapped(small_kernel<NT, 2, kQ8>, dim3(grid), dim3(256), 0, s, p);
    case 4: return launch_overlapped(small_kernel<NT, 4, kQ8>, dim3(grid), dim3(256), 0, s, p);
    default: return launch_overlapped(small_kernel<NT, 8, kQ8>, dim3(grid), dim3(256), 0, s, p);
  }
}

template <bool kQ8>
cudaError_t launch_small(const SmallParams& p, int num_sms, cudaStream_t s) {
  prof::Scope scope(kQ8 ? "linear_small_q8" : "linear_small", s);
  if (p.T <= 8) return launch_small_nt<1, kQ8>(p, num_sms, s);
  if (p.T <= 16) return launch_small_nt<2, kQ8>(p, num_sms, s);
  return launch_small_nt<4, kQ8>(p, num_sms, s);
}

// ------------------------------------------------------------ entry points
moe_status check_call(moe_linear* L, int T, int most) {
  if (!L) return fail(MOE_ERR_INVALID, "linear is NULL");
  if (T < 1 || T > L->cfg.max_tokens || T > most)
    return fail(MOE_ERR_CAPACITY, "n_tokens=%d outside [1, %d]", T, min(L->cfg.max_tokens, most));
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != L->device) return fail(MOE_ERR_INVALID, "the handle belongs to device %d, not %d", L->device, dev);
  return MOE_OK;
}

moe_status check_io(const Buf* in, int n_in, const Buf& y, int dev) {
  moe_status st;
  for (int i = 0; i < n_in; ++i) {
    if ((st = check_buf(in[i], dev)) != MOE_OK) return st;
    if (overlap(in[i], y)) return fail(MOE_ERR_INVALID, "y overlaps %s", in[i].name);
  }
  return check_buf(y, dev);
}

moe_status create(const moe_linear_config* c, const moe_linear_weights* w, int on_device, moe_linear** out) {
  if (!out) return fail(MOE_ERR_INVALID, "out is NULL");
  *out = nullptr;
  if (!c) return fail(MOE_ERR_INVALID, "config is NULL");
  if (c->in_features < 32 || c->in_features > 32768 || c->in_features % 32)
    return fail(MOE_ERR_INVALID, "in_features=%d: a multiple of 32 in [32, 32768] is needed", c->in_features);
  if (c->out_features < 1 || c->out_features > (1 << 20))
    return fail(MOE_ERR_INVALID, "out_features=%d outside [1, %d]", c->out_features, 1 << 20);
  if (c->max_tokens < 1 || c->max_tokens > 65536)
    return fail(MOE_ERR_INVALID, "max_tokens=%d outside [1, 65536]", c->max_tokens);
  if (!w || !w->q || !w->s) return fail(MOE_ERR_INVALID, "a required weight pointer is NULL");
  moe_linear* L = new (std::nothrow) moe_linear();
  if (!L) return fail(MOE_ERR_OOM, "out of host memory");
  L->cfg = *c;
  cudaError_t e = cudaGetDevice(&L->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&L->num_sms, cudaDevAttrMultiProcessorCount, L->device);
  if (e != cudaSuccess) {
    delete L;
    return cuda_fail(e, "query the device");
  }
  const int N = c->out_features, K = c->in_features;
  L->w.N = N;
  L->w.K = K;
  L->w.kc = (K + kTileK - 1) / kTileK;
  L->w.nt = (N + kTileRows - 1) / kTileRows;
  const size_t n_tiles = (size_t)L->w.nt * L->w.kc, tiles = n_tiles * kTileBytes;
  const size_t o_bias = (tiles + 255) & ~(size_t)255, o_err = o_bias + (((size_t)N * 4 + 255) & ~(size_t)255);
  const size_t qb = (size_t)N * (K / 2), sb = (size_t)N * (K / 32) * 2;
  void* tmp = nullptr;  // device copies of host weights while they are packed
  auto bad = [&](cudaError_t err, const char* what) {
    cudaFree(tmp);
    moe_linear_destroy(L);
    return cuda_fail(err, what);
  };
  if ((e = cudaMalloc(&L->block, o_err + 256)) != cudaSuccess) return bad(e, "cudaMalloc(linear weights)");
  char* base = static_cast<char*>(L->block);
  L->w.tiles = reinterpret_cast<const uint8_t*>(base);
  L->w.bias = w->bias ? reinterpret_cast<const float*>(base + o_bias) : nullptr;
  L->err = reinterpret_cast<int*>(base + o_err);
  const uint8_t* q = w->q;
  const uint16_t* s = w->s;
  if (!on_device) {
    const size_t qa = (qb + 255) & ~(size_t)255;
    if ((e = cudaMalloc(&tmp, qa + sb)) != cudaSuccess) return bad(e, "cudaMalloc(weight staging)");
    if ((e = cudaMemcpy(tmp, w->q, qb, cudaMemcpyHostToDevice)) != cudaSuccess) return bad(e, "copy codes");
    if ((e = cudaMemcpy(static_cast<char*>(tmp) + qa, w->s, sb, cudaMemcpyHostToDevice)) != cudaSuccess)
      return bad(e, "copy scales");
    q = static_cast<const uint8_t*>(tmp);
    s = reinterpret_cast<const uint16_t*>(static_cast<char*>(tmp) + qa);
  }
  // device sources may still be written by the caller's streams
  if ((e = cudaDeviceSynchronize()) != cudaSuccess) return bad(e, "cudaDeviceSynchronize");
  pack_kernel<<<(unsigned)((n_tiles + 7) / 8), 256>>>(q, s, N, K, L->w.kc, reinterpret_cast<uint8_t*>(base));
  if ((e = cudaGetLastError()) != cudaSuccess) return bad(e, "pack weights");
  if (w->bias && (e = cudaMemcpy(base + o_bias, w->bias, (size_t)N * 4,
                                 on_device ? cudaMemcpyDeviceToDevice : cudaMemcpyHostToDevice)) != cudaSuccess)
    return bad(e, "copy bias");
  if ((e = cudaMemset(base + o_err, 0, 256)) != cudaSuccess) return bad(e, "clear the error word");
  if ((e = cudaDeviceSynchronize()) != cudaSuccess) return bad(e, "pack weights");
  cudaFree(tmp);
  *out = L;
  return MOE_OK;
}

moe_status forward(moe_linear* L, const void* x, int T, void* y, void* stream) {
  moe_status st = check_call(L, T, 65536);
  if (st != MOE_OK) return st;
  const int K = L->w.K, N = L->w.N;
  const Buf in[1] = {{"x", x, (size_t)T * K * 2, 16}};
  if ((st = check_io(in, 1, Buf{"y", y, (size_t)T * N * 2, 2}, L->device)) != MOE_OK) return st;
  SmallParams p = {};
  p.w = L->w;
  for (int t = 0; t < T; t += 32) {
    p.T = min(32, T - t);
    p.x = static_cast<const uint16_t*>(x) + (size_t)t * K;
    p.y = static_cast<uint16_t*>(y) + (size_t)t * N;
    const cudaError_t e = launch_small<false>(p, L->num_sms, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "linear launch");
  }
  return MOE_OK;
}

moe_status forward_q8(moe_linear* L, const int8_t* q, const float* qs, int T, void* y, void* stream) {
  moe_status st = check_call(L, T, kMaxQ8Tokens);
  if (st != MOE_OK) return st;
  const int K = L->w.K, N = L->w.N;
  const Buf in[2] = {{"x_q8", q, (size_t)T * K, 16}, {"x_scale", qs, (size_t)T * (K / 32) * 4, 4}};
  if ((st = check_io(in, 2, Buf{"y", y, (size_t)T * N * 2, 2}, L->device)) != MOE_OK) return st;
  SmallParams p = {};
  p.w = L->w;
  p.T = T;
  p.q = q;
  p.qs = qs;
  p.y = static_cast<uint16_t*>(y);
  const cudaError_t e = launch_small<true>(p, L->num_sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "linear launch");
  return MOE_OK;
}

}  // namespace
}  // namespace lin
}  // namespace moe

extern "C" {

moe_status moe_linear_create(const moe_linear_config* cfg, const moe_linear_weights* w, int weights_on_device,
                             moe_linear** out) {
  return moe::lin::create(cfg, w, weights_on_device, out);
}

void moe_linear_destroy(moe_linear* linear) {
  if (!linear) return;
  cudaDeviceSynchronize();
  if (linear->block) cudaFree(linear->block);
  cudaGetLastError();
  delete linear;
}

moe_status moe_linear_forward(moe_linear* linear, const void* x_bf16, int n_tokens, void* y_bf16, void* stream) {
  return moe::lin::forward(linear, x_bf16, n_tokens, y_bf16, stream);
}

moe_status moe_linear_forward_q8(moe_linear* linear, const int8_t* x_q8, const float* x_scale, int n_tokens,
                                 void* y_bf16, void* stream) {
  return moe::lin::forward_q8(linear, x_q8, x_scale, n_tokens, y_bf16, stream);
}

moe_status moe_linear_status_sync(moe_linear* linear, void* stream) {
  using namespace moe::op;
  if (!linear) return fail(MOE_ERR_INVALID, "linear is NULL");
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int err = 0;
  if ((e = cudaMemcpy(&err, linear->err, sizeof err, cudaMemcpyDeviceToHost)) != cudaSuccess)
    return cuda_fail(e, "read error word");
  if (err != 0) {
    if ((e = cudaMemset(linear->err, 0, sizeof err)) != cudaSuccess) return cuda_fail(e, "clear error word");
    return fail((moe_status)err, "a kernel recorded error %d", err);
  }
  return MOE_OK;
}

}  // extern "C"
