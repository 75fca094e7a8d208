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
#include <stdlib.h>

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
// Per row: the power of two that brings the largest |scale| to [2^15, 2^16)
// (shift) and row_f = 2^-shift.  A row with an infinite or NaN scale, or with
// none but zeros, keeps its scales.
__global__ void row_shift_kernel(const uint16_t* __restrict__ s, int N, int nb, float* __restrict__ row_f) {
  const int row = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= N) return;
  uint32_t m = 0;
  for (int i = lane; i < nb; i += 32) m = max(m, (uint32_t)(s[(size_t)row * nb + i] & 0x7fffu));
  for (int k = 16; k >= 1; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
  if (lane == 0) {
    const float v = __half2float(__ushort_as_half((uint16_t)m));
    const int e = (m == 0 || m >= 0x7c00u) ? 15 : ilogbf(v);
    row_f[row] = pow2f(e - 15);
  }
}

// One warp per tile.
__global__ void pack_kernel(const uint8_t* __restrict__ q, const uint16_t* __restrict__ s, int N, int K, int kc,
                            const float* __restrict__ row_f, uint8_t* __restrict__ tiles) {
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
      uint32_t c[8] = {8, 8, 8, 8, 8, 8, 8, 8};  // weight 0
      if (row < N && k < K) {
        const uint8_t* b = q + (size_t)row * (K / 2) + k / 2;  // four bytes: inputs k .. k + 7
        for (int j = 0; j < 4; ++j) c[2 * j] = b[j] & 15, c[2 * j + 1] = b[j] >> 4;
      }
      w[i] = word_of(c);
    }
    *reinterpret_cast<uint4*>(dst + 512 * half + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  for (int i = lane; i < 64; i += 32) {  // scale i: 8 g' + (0..3 row g', 4..7 row g' + 8)
    const int row = row0 + (i >> 3) + 8 * ((i >> 2) & 1), blk = k0 / 32 + (i & 3);
    uint16_t v = 0;
    if (row < N && blk < K / 32)
      v = __half_as_ushort(__float2half_rn(__half2float(__ushort_as_half(s[(size_t)row * (K / 32) + blk])) / row_f[row]));
    reinterpret_cast<uint16_t*>(dst + kTileCodes)[i] = v;
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

// D = A B + C, A 16x16 (rows x inputs), B 16x8 (inputs x tokens), bf16 -> fp32
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Pair i of a word as bf16 integers code - 8: a 4-bit code ORed into bits 3-6
// of 16.0 reads 16 + code, and the difference to 24 is exact.  (Taking the
// offset off in the accumulator instead, with an MMA of constant -24 for
// operand A, saves 8 instructions per lane and block but is slower: these
// kernels wait for the legacy MMA pipe first.)
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int i) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
      : "=r"(v)
      : "r"(i == 3 ? __funnelshift_r(w, w, 12) : w >> (4 * i)), "r"(0x00780078u), "r"(0x41804180u));
  const __nv_bfloat162 k24 = __halves2bfloat162(__ushort_as_bfloat16(0x41C0), __ushort_as_bfloat16(0x41C0));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), k24);
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Four signed bytes as two words of bf16 pairs (exact).  With 0x43 above it a
// byte's low seven bits read 128 + (c & 127), and its sign bit alone 128 or,
// set, 256: the difference is the signed value.
__device__ __forceinline__ void bytes_to_bf16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = __byte_perm(c, 0x43434343u, i ? 0x4342u : 0x4140u);
    const uint32_t m = v & 0xff7fff7fu, n = v & 0xff80ff80u;
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&n));
    o[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
  lo = o[0];
  hi = o[1];
}

// The inputs of one scale block as a lane of a B fragment holds them: eight
// consecutive inputs of token 8 n + g (and the scales of tokens 8 n + 2 t, + 1).
template <int NT, bool kQ8>
struct XBlock {
  uint4 c[NT];
};
template <int NT>
struct XBlock<NT, true> {
  uint2 c[NT];
  float f[NT][2];
};

// CTAs of 8 warps; a unit is MT 16-row tiles, shared by S warps that take a
// contiguous part of the K tiles each (their partial sums meet in shared
// memory, in one fixed order).  A warp streams its weights through a ring of
// its own of ST stages in shared memory (16-byte asynchronous copies, no
// barrier between warps); x comes through L1.
template <int NT, int MT, int ST, int kCtas, bool kQ8>
__global__ void __launch_bounds__(256, kCtas) small_kernel(const __grid_constant__ SmallParams p, int S) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kStage = MT * kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  unsigned char* ring = smem + warp * ST * kStage;
  float* part = reinterpret_cast<float*>(smem + 8 * ST * kStage);
  const int kc = p.w.kc, K = p.w.K;
  const int ks = warp % S, grp = warp / S;
  const int c0 = ks * kc / S, c1 = (ks + 1) * kc / S;
  const int units = (p.w.nt + MT - 1) / MT;
  const int ustep = gridDim.x * (8 / S);
  const int unit0 = blockIdx.x * (8 / S) + grp;

  // Next stage to fill: unit, K tile, this lane's source and destination.
  // Tiles of a unit past the end are the last tile again (not stored).
  int lu = unit0, lc = c0;
  const uint8_t* lsrc = p.w.tiles;
  uint32_t ldst = smem_u32(ring) + 16 * lane;
  const uint32_t lend = ldst + ST * kStage;
  uint32_t mstep[MT];
  auto source = [&]() {
    const int tile = min(lu * MT, p.w.nt - 1);
    lsrc = p.w.tiles + ((size_t)tile * kc + c0) * kTileBytes + 16 * lane;
#pragma unroll
    for (int m = 0; m < MT; ++m) mstep[m] = (uint32_t)(min(m, p.w.nt - 1 - tile) * kc * kTileBytes);
  };
  source();
  auto issue = [&]() {
    if (lu < units) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint8_t* src = lsrc + mstep[m];
        cp_async_16(ldst + m * kTileBytes, src);
        cp_async_16(ldst + m * kTileBytes + 512, src + 512);
        if (lane < 8) cp_async_16(ldst + m * kTileBytes + kTileCodes, src + kTileCodes);
      }
      lsrc += kTileBytes;
      if (++lc == c1) {
        lc = c0;
        lu += ustep;
        source();
      }
    }
    cp_async_commit();
    ldst += kStage;
    if (ldst == lend) ldst -= ST * kStage;
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) issue();  // the weights are the library's own: nothing to wait for
  dep_wait();
  dep_release();

  // x: lanes of tokens past the batch read the last token (their columns are
  // not stored), inputs past K the last block (their scales are zero), so no
  // load needs a predicate.  Block b + 1 is loaded before block b is used.
  int xo[NT], so[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xo[n] = min(8 * n + g, p.T - 1) * K + 8 * t;
    so[n][0] = min(8 * n + 2 * t, p.T - 1) * (K >> 5);
    so[n][1] = min(8 * n + 2 * t + 1, p.T - 1) * (K >> 5);
  }
  XBlock<NT, kQ8> xb[2];
  auto load_x = [&](XBlock<NT, kQ8>& v, int k) {
    k = min(k, K - 32);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (kQ8) {
        v.c[n] = *reinterpret_cast<const uint2*>(p.q + xo[n] + k);
        v.f[n][0] = p.qs[so[n][0] + (k >> 5)];
        v.f[n][1] = p.qs[so[n][1] + (k >> 5)];
      } else {
        v.c[n] = *reinterpret_cast<const uint4*>(p.x + xo[n] + k);
      }
    }
  };
  load_x(xb[0], c0 * kTileK);

  int slot = 0;
  for (int unit = unit0; unit - grp < units; unit += ustep) {  // the same number of turns for every warp
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
    if (unit < units) {
      for (int c = c0; c < c1; ++c) {
        cp_async_wait<ST - 2>();
        __syncwarp();  // the stage is there for every lane, and every lane is done with the one before
        issue();
        const unsigned char* st = ring + slot * kStage;
        slot = slot + 1 == ST ? 0 : slot + 1;
        uint4 sc[MT], wv[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          sc[m] = *reinterpret_cast<const uint4*>(st + m * kTileBytes + kTileCodes + 16 * g);
        const int kn = (c + 1 < c1 ? c + 1 : c0) * kTileK;  // the next stage's first input
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          load_x(xb[(b + 1) & 1], b < 3 ? c * kTileK + 32 * (b + 1) : kn);
          XBlock<NT, kQ8>& xc = xb[b & 1];
          uint4 xv[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (kQ8) {
              bytes_to_bf16(xc.c[n].x, xv[n].x, xv[n].y);
              bytes_to_bf16(xc.c[n].y, xv[n].z, xv[n].w);
            } else {
              xv[n] = xc.c[n];
            }
          }
          if ((b & 1) == 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
              wv[m] = *reinterpret_cast<const uint4*>(st + m * kTileBytes + 512 * (b >> 1) + 16 * lane);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint2 w = (b & 1) ? make_uint2(wv[m].z, wv[m].w) : make_uint2(wv[m].x, wv[m].y);
            const uint32_t s0 = (b >> 1) ? sc[m].y : sc[m].x, s1 = (b >> 1) ? sc[m].w : sc[m].z;
            const __half2 h0 = *reinterpret_cast<const __half2*>(&s0), h1 = *reinterpret_cast<const __half2*>(&s1);
            const float sg = (b & 1) ? __high2float(h0) : __low2float(h0);
            const float sh = (b & 1) ? __high2float(h1) : __low2float(h1);
            uint32_t a0[4], a1[4];
            float dn[NT][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a0[i] = unpack_pair(w.x, i);
              a1[i] = unpack_pair(w.y, i);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_bf16(dn[n], a0[0], a1[0], a0[1], a1[1], xv[n].x, xv[n].y, 0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_bf16(dn[n], a0[2], a1[2], a0[3], a1[3], xv[n].z, xv[n].w, dn[n][0], dn[n][1], dn[n][2], dn[n][3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float (&d)[4] = dn[n];
              if constexpr (kQ8) {
                d[0] *= xc.f[n][0], d[1] *= xc.f[n][1], d[2] *= xc.f[n][0], d[3] *= xc.f[n][1];
              }
              acc[m][n][0] = fmaf(sg, d[0], acc[m][n][0]);
              acc[m][n][1] = fmaf(sg, d[1], acc[m][n][1]);
              acc[m][n][2] = fmaf(sh, d[2], acc[m][n][2]);
              acc[m][n][3] = fmaf(sh, d[3], acc[m][n][3]);
            }
          }
        }
      }
    }
    if (S > 1) {
      __syncthreads();  // the sums of the unit before are read
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<float4*>(&part[(((warp * MT + m) * NT + n) * 32 + lane) * 4]) =
              make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
      __syncthreads();
      if (ks == 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            for (int i = 1; i < S; ++i) {
              const float4 v =
                  *reinterpret_cast<const float4*>(&part[((((warp + i) * MT + m) * NT + n) * 32 + lane) * 4]);
              acc[m][n][0] += v.x, acc[m][n][1] += v.y, acc[m][n][2] += v.z, acc[m][n][3] += v.w;
            }
      }
    }
    if (unit < units && ks == 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = (unit * MT + m) * kTileRows + g + 8 * h;
          if (row < p.w.N) {
            const float rf = __ldg(p.w.row_f + row), bias = p.w.bias ? __ldg(p.w.bias + row) : 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int tok = 8 * n + 2 * t + i;
                if (tok < p.T)
                  p.y[(size_t)tok * p.w.N + row] =
                      __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(acc[m][n][2 * h + i], rf, bias)));
              }
          }
        }
    }
  }
  cp_async_wait<0>();  // (only empty groups are left)
}

template <int NT, int MT, int ST, int kCtas, bool kQ8>
cudaError_t launch_small_as(const SmallParams& p, int num_sms, cudaStream_t s) {
  constexpr int kRing = 8 * ST * MT * kTileBytes, kPart = 8 * MT * NT * 512;
  static const cudaError_t attr =
      cudaFuncSetAttribute(small_kernel<NT, MT, ST, kCtas, kQ8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + kPart);
  if (attr != cudaSuccess) return attr;
  // Warps per unit: the smallest power of two whose last round of units
  // leaves at most 1/16 of the warps idle, else the one that leaves fewest.
  const int units = (p.w.nt + MT - 1) / MT, slots = 8 * kCtas * num_sms;
  int S = 1;
  double best = 0.0;
  for (int c = 1; c <= 8 && c <= p.w.kc; c *= 2) {
    const int rounds = (units * c + slots - 1) / slots;
    const double used = (double)units * c / ((double)rounds * slots);
    if (used > best) S = c, best = used;
    if (best > 0.9375) break;
  }
  const int per = 8 / S;
  const int grid = min((units + per - 1) / per, kCtas * num_sms);
  return launch_overlapped(small_kernel<NT, MT, ST, kCtas, kQ8>, dim3(grid), dim3(256), kRing + (S > 1 ? kPart : 0), s, p, S);
}

template <bool kQ8>
cudaError_t launch_small(const SmallParams& p, int num_sms, cudaStream_t s) {
  prof::Scope scope(kQ8 ? "linear_small_q8" : "linear_small", s);
  static const int v = getenv("LV") ? atoi(getenv("LV")) : 0;
  if (p.T <= 8) {
    if (v == 1) return launch_small_as<1, 1, 6, 3, kQ8>(p, num_sms, s);
    if (v == 2) return launch_small_as<1, 2, 4, 2, kQ8>(p, num_sms, s);
    if (v == 3) return launch_small_as<1, 1, 4, 4, kQ8>(p, num_sms, s);
    if (v == 4) return launch_small_as<1, 2, 3, 3, kQ8>(p, num_sms, s);
    return launch_small_as<1, 1, 8, 2, kQ8>(p, num_sms, s);
  }
  if (p.T <= 16) {
    if (v == 1) return launch_small_as<2, 1, 6, 2, kQ8>(p, num_sms, s);
    if (v == 2) return launch_small_as<2, 2, 5, 1, kQ8>(p, num_sms, s);
    return launch_small_as<2, 2, 4, 2, kQ8>(p, num_sms, s);
  }
  if (v == 1) return launch_small_as<4, 4, 4, 1, kQ8>(p, num_sms, s);
  if (v == 2) return launch_small_as<4, 2, 6, 1, kQ8>(p, num_sms, s);
  return launch_small_as<4, 2, 4, 2, kQ8>(p, num_sms, s);
}

// ------------------------------------------------------------ entry points
moe_status check_call(moe_linear* L, int T) {
  if (!L) return fail(MOE_ERR_INVALID, "linear is NULL");
  if (T < 1 || T > L->cfg.max_tokens)
    return fail(MOE_ERR_CAPACITY, "n_tokens=%d outside [1, %d]", T, L->cfg.max_tokens);
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
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  const size_t o_rf = up(tiles), o_bias = o_rf + up((size_t)N * 4), o_err = o_bias + up((size_t)N * 4), o_ws = o_err + 256;
  const size_t qb = (size_t)N * (K / 2), sb = (size_t)N * (K / 32) * 2;
  void* tmp = nullptr;  // device copies of host weights while they are packed
  auto bad = [&](cudaError_t err, const char* what) {
    cudaFree(tmp);
    moe_linear_destroy(L);
    return cuda_fail(err, what);
  };
  if ((e = cudaMalloc(&L->block, o_ws + gemm_workspace(K, c->max_tokens))) != cudaSuccess) return bad(e, "cudaMalloc(linear weights)");
  char* base = static_cast<char*>(L->block);
  L->w.tiles = reinterpret_cast<const uint8_t*>(base);
  L->w.row_f = reinterpret_cast<const float*>(base + o_rf);
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
  row_shift_kernel<<<(N + 7) / 8, 256>>>(s, N, K / 32, reinterpret_cast<float*>(base + o_rf));
  pack_kernel<<<(unsigned)((n_tiles + 7) / 8), 256>>>(q, s, N, K, L->w.kc, L->w.row_f, reinterpret_cast<uint8_t*>(base));
  if ((e = cudaGetLastError()) != cudaSuccess) return bad(e, "pack weights");
  if (w->bias && (e = cudaMemcpy(base + o_bias, w->bias, (size_t)N * 4,
                                 on_device ? cudaMemcpyDeviceToDevice : cudaMemcpyHostToDevice)) != cudaSuccess)
    return bad(e, "copy bias");
  if ((e = cudaMemset(base + o_err, 0, 256)) != cudaSuccess) return bad(e, "clear the error word");
  if ((e = cudaDeviceSynchronize()) != cudaSuccess) return bad(e, "pack weights");
  cudaFree(tmp);
  moe_status st = gemm_init(L, base + o_ws);
  if (st != MOE_OK) {
    moe_linear_destroy(L);
    return st;
  }
  *out = L;
  return MOE_OK;
}

moe_status run(moe_linear* L, const XIn& in, int T, void* y, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  if (T > kSmallTokens) return launch_gemm(L, in, T, static_cast<uint16_t*>(y), s);
  SmallParams p = {};
  p.w = L->w;
  p.T = T;
  p.x = in.x;
  p.q = in.q;
  p.qs = in.qs;
  p.y = static_cast<uint16_t*>(y);
  const cudaError_t e = in.x ? launch_small<false>(p, L->num_sms, s) : launch_small<true>(p, L->num_sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "linear launch");
  return MOE_OK;
}

moe_status forward(moe_linear* L, const void* x, int T, void* y, void* stream) {
  moe_status st = check_call(L, T);
  if (st != MOE_OK) return st;
  const int K = L->w.K, N = L->w.N;
  const Buf in[1] = {{"x", x, (size_t)T * K * 2, 16}};
  if ((st = check_io(in, 1, Buf{"y", y, (size_t)T * N * 2, 2}, L->device)) != MOE_OK) return st;
  return run(L, XIn{static_cast<const uint16_t*>(x), nullptr, nullptr}, T, y, stream);
}

moe_status forward_q8(moe_linear* L, const int8_t* q, const float* qs, int T, void* y, void* stream) {
  moe_status st = check_call(L, T);
  if (st != MOE_OK) return st;
  const int K = L->w.K, N = L->w.N;
  const Buf in[2] = {{"x_q8", q, (size_t)T * K, 16}, {"x_scale", qs, (size_t)T * (K / 32) * 4, 4}};
  if ((st = check_io(in, 2, Buf{"y", y, (size_t)T * N * 2, 2}, L->device)) != MOE_OK) return st;
  return run(L, XIn{nullptr, q, qs}, T, y, stream);
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
