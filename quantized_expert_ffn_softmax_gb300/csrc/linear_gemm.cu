// moe_linear on batches above kSmallTokens: tcgen05 GEMM with the 4-bit
// weights dequantised on the way into shared memory.
//
//   prep   x (bf16, or 8-bit codes with scales) -> x16: fp16, every token
//          scaled by a power of two so that its largest magnitude lies in
//          [1, 2) (bf16 values keep all their bits down to 2^-14 of that)
//   gemm   D[128 rows of W x BN tokens] = W' x16^T in TMEM, fp32; epilogue
//          y = D * row factor * token factor + bias, one rounding to bf16
//
// W' = (code - 8) * s' is rounded once to fp16 (relative 2^-12): a code in
// bits 3-6 of a zero half word reads code * 2^-21 (an fp16 subnormal), so one
// fp16 FMA with s = s' * 2^21, which is how the scales are stored, and -8 s'
// gives the weight with a single rounding.
//
// One CTA per SM, warp-specialised.  Warps 0-3: epilogue.  Warps 4-11:
// producers, each streams the tiles of its own 16 rows through a ring of its
// own (16-byte asynchronous copies) and writes fp16 rows into the stage's A
// tile (128-byte swizzle, K-major).  Warp 12: TMA of the x16 tile.  Warp 13:
// MMA issue.  Few row blocks: S CTAs of a cluster share one output tile, each
// with a part of K, and sum their fp32 tiles through distributed shared
// memory in rank order.
#include <string.h>

#include <algorithm>

#include "device_common.cuh"
#include "linear_internal.cuh"
#include "op_common.cuh"
#include "profile.cuh"

namespace moe {
namespace lin {
namespace {

using namespace dev;
using namespace op;

constexpr int kRowsA = 128;               // rows of W per tile
constexpr int kStepK = 64;                // inputs per stage
constexpr int kABytes = kRowsA * 128;     // A tile of a stage
constexpr int kProdWarps = 8;
constexpr int kLoadWarp = 4 + kProdWarps;
constexpr int kMmaWarp = kLoadWarp + 1;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kRing = 6;                  // packed tiles in flight per producer warp
constexpr int kRingBytes = kProdWarps * kRing * kTileBytes;
constexpr int kMaxStages = 8;
constexpr int kBarBytes = 256;
constexpr int kMaxSmem = 227 * 1024;

// ------------------------------------------------------------ prep
template <bool kQ8, int V>
__global__ void __launch_bounds__(1024) prep_kernel(const XIn in, int K, __half* __restrict__ x16,
                                                    float* __restrict__ x_f) {
  __shared__ uint32_t red[32];
  dep_wait();
  dep_release();
  const int t = blockIdx.x, nvec = K >> 3;
  float v[V][8];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] = 0.0f;
    if (i < nvec) {
      if constexpr (kQ8) {
        const int2 c = *reinterpret_cast<const int2*>(in.q + (size_t)t * K + 8 * i);
        const float f = in.qs[(size_t)t * (K >> 5) + (i >> 2)];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] = f * (float)(int8_t)((k < 4 ? c.x : c.y) >> (8 * (k & 3)));
      } else {
        const uint4 c = *reinterpret_cast<const uint4*>(in.x + (size_t)t * K + 8 * i);
        v[j][0] = bf_lo(c.x), v[j][1] = bf_hi(c.x), v[j][2] = bf_lo(c.y), v[j][3] = bf_hi(c.y);
        v[j][4] = bf_lo(c.z), v[j][5] = bf_hi(c.z), v[j][6] = bf_lo(c.w), v[j][7] = bf_hi(c.w);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[j][k]) & 0x7fffffffu);
  }
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0u;
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
  // exponent of the largest magnitude; a token with an infinity or NaN, or of
  // zeros only, is left as it is
  const int e = (m == 0 || m >= 0x7f800000u) ? 0 : max(-126, min(126, (int)(m >> 23) - 127));
  const float f = pow2f(-e);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    if (i < nvec) {
      __half2 h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = __floats2half2_rn(v[j][2 * k] * f, v[j][2 * k + 1] * f);
      *reinterpret_cast<uint4*>(x16 + (size_t)t * K + 8 * i) = *reinterpret_cast<const uint4*>(h);
    }
  }
  if (threadIdx.x == 0) x_f[t] = pow2f(e);
}

// ------------------------------------------------------------ gemm
struct GemmParams {
  Weights w;
  const float* x_f;
  uint16_t* y;
  int T;
  int bn;        // tokens per tile: a multiple of 16, 16 .. 256
  int n_rb;      // row blocks
  int units;     // row blocks x token tiles
  int split;     // CTAs of a cluster that share a unit (1: units are walked persistently)
  int stages;
  int tmem_cols;
  int* err;
  unsigned long long timeout_ns;
};

// Word of 8 codes -> 8 weights (code - 8) s' as fp16, in input order.
// s: the stored scale s' 2^21 in both halves, c: -8 s'.
__device__ __forceinline__ uint4 dequant8(uint32_t w, __half2 s, __half2 c) {
  uint32_t v[4] = {w & 0x00780078u, (w >> 4) & 0x00780078u, (w >> 8) & 0x00780078u,
                   __funnelshift_r(w, w, 12) & 0x00780078u};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&v[i]), s, c);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t saddr, int rank) {
  float v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}\n"
      : "=f"(v)
      : "r"(saddr), "r"(rank)
      : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  const int bn = p.bn, S = p.stages;
  const int stage_bytes = kABytes + bn * 128;
  unsigned char* ring0 = smem + S * stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring0 + kRingBytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* tdrain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdrain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], kProdWarps + 1);  // + the loader's arrive with the tile's bytes
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4 * 32);
    }
    mbar_init(tdrain, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tmo = p.timeout_ns;

  // this CTA's units, and its part of K in packed tiles (128 inputs) and steps
  const int split = p.split, rank = split > 1 ? (int)(blockIdx.x % split) : 0;
  const int u0 = blockIdx.x / split, ustep = split > 1 ? p.units : gridDim.x;
  const int kc = p.w.kc;
  const int c0 = rank * kc / split, c1 = (rank + 1) * kc / split;
  const int steps = min(2 * c1, (p.w.K + kStepK - 1) / kStepK) - 2 * c0;

  if (warp < 4) {
    // ------------------------------------------------------------ epilogue
    // Thread r owns row r of the tile (TMEM lane r).
    dep_wait();
    dep_release();
    const int r = warp * 32 + lane;
    int j = 0;
    for (int u = u0; u < p.units; u += ustep, ++j) {
      const int row = (u % p.n_rb) * kRowsA + r, t0 = (u / p.n_rb) * bn;
      const int nt = min(bn, p.T - t0);
      const int b = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[b], (j >> 1) & 1, p.err, tmo))) break;
      tc_fence_after();
      const uint32_t tb = tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(b * bn);
      if (split == 1) {
        const bool in = row < p.w.N;
        const float rf = in ? __ldg(p.w.row_f + row) * 0x1p21f : 0.0f;
        const float bias = in && p.w.bias ? __ldg(p.w.bias + row) : 0.0f;
        for (int c = 0; c < nt; c += 16) {
          uint32_t v[16];
          tmem_ld16(tb + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = t0 + c + i;
            if (in && c + i < nt)
              p.y[(size_t)t * p.w.N + row] = __bfloat16_as_ushort(
                  __float2bfloat16_rn(fmaf(__uint_as_float(v[i]) * rf, p.x_f[t], bias)));
          }
        }
      } else {
        // the tile as [token][128 rows] fp32 over the stages (all MMAs are done)
        float* part = reinterpret_cast<float*>(smem);
        for (int c = 0; c < nt; c += 16) {
          uint32_t v[16];
          tmem_ld16(tb + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(c + i) * kRowsA + r] = __uint_as_float(v[i]);
        }
      }
      tc_fence_before();
      mbar_arrive(&tempty[b]);
    }
  } else if (warp < kLoadWarp) {
    // ------------------------------------------------------------ producers
    const int w = warp - 4, g = lane >> 2, t = lane & 3;
    unsigned char* ring = ring0 + w * kRing * kTileBytes;
    int lu = u0, lc = c0;
    const uint8_t* lsrc = nullptr;
    auto source = [&]() {
      const int tile = min((lu % p.n_rb) * (kRowsA / kTileRows) + w, p.w.nt - 1);  // past N: not stored
      lsrc = p.w.tiles + ((size_t)tile * kc + c0) * kTileBytes + 16 * lane;
    };
    source();
    uint32_t ldst = smem_u32(ring) + 16 * lane;
    const uint32_t lend = ldst + kRing * kTileBytes;
    auto issue = [&]() {
      if (lu < p.units) {
        cp_async_16(ldst, lsrc);
        cp_async_16(ldst + 512, lsrc + 512);
        if (lane < 8) cp_async_16(ldst + kTileCodes, lsrc + kTileCodes);
        lsrc += kTileBytes;
        if (++lc == c1) {
          lc = c0;
          lu += ustep;
          source();
        }
      }
      cp_async_commit();
      ldst += kTileBytes;
      if (ldst == lend) ldst -= kRing * kTileBytes;
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue();  // the weights are the library's own: nothing to wait for
    dep_wait();
    dep_release();
    int slot = 0, st = 0;
    uint32_t par = 1;  // parity of the stage's next "empty" phase
    bool alive = true;
    // rows g and g + 8 of the warp's 16: 16-byte chunk 4 b + t of the row for
    // block b, XOR-swizzled by the row; odd rows store their blocks in the
    // other order, so that eight lanes touch eight different chunks
    const uint32_t a_row = (uint32_t)((16 * w + g) * 128);
    const uint32_t o0 = a_row + (uint32_t)(((4 * (g & 1) + t) ^ g) * 16);
    const uint32_t o1 = a_row + (uint32_t)(((4 * ((g & 1) ^ 1) + t) ^ g) * 16);
    for (int u = u0; u < p.units && alive; u += ustep) {
      for (int s2 = 0; s2 < steps && alive; s2 += 2) {
        cp_async_wait<kRing - 2>();
        __syncwarp();  // the tile is there for every lane, and every lane is done with the one before
        issue();
        const unsigned char* tl = ring + slot * kTileBytes;
        slot = slot + 1 == kRing ? 0 : slot + 1;
        const uint4 sc = *reinterpret_cast<const uint4*>(tl + kTileCodes + 16 * g);
        const __half2 k8 = __half2half2(__ushort_as_half(0x8040));  // -2^-18
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (s2 + h >= steps) break;
          const uint4 wd = *reinterpret_cast<const uint4*>(tl + 512 * h + 16 * lane);
          const uint32_t s0 = h ? sc.y : sc.x, s1 = h ? sc.w : sc.z;
          const __half2 q0 = *reinterpret_cast<const __half2*>(&s0), q1 = *reinterpret_cast<const __half2*>(&s1);
          const __half2 a0 = __low2half2(q0), a1 = __high2half2(q0), b0 = __low2half2(q1), b1 = __high2half2(q1);
          const uint4 r00 = dequant8(wd.x, a0, __hmul2(a0, k8)), r80 = dequant8(wd.y, b0, __hmul2(b0, k8));
          const uint4 r01 = dequant8(wd.z, a1, __hmul2(a1, k8)), r81 = dequant8(wd.w, b1, __hmul2(b1, k8));
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], par, p.err, tmo))) {
            alive = false;
            break;
          }
          unsigned char* A = smem + st * stage_bytes;
          const bool odd = g & 1;
          *reinterpret_cast<uint4*>(A + o0) = odd ? r01 : r00;
          *reinterpret_cast<uint4*>(A + o0 + 1024) = odd ? r81 : r80;
          *reinterpret_cast<uint4*>(A + o1) = odd ? r00 : r01;
          *reinterpret_cast<uint4*>(A + o1 + 1024) = odd ? r80 : r81;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[st]);
          if (++st == S) st = 0, par ^= 1;
        }
      }
    }
    cp_async_wait<0>();
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ x16 tiles
    dep_wait();
    dep_release();
    int st = 0;
    uint32_t par = 1, n = 0;
    bool alive = true;
    for (int u = u0; u < p.units && alive; u += ustep) {
      const int t0 = (u / p.n_rb) * bn;
      for (int s = 0; s < steps; ++s, ++n) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], par, p.err, tmo))) {
          alive = false;
          break;
        }
        if (elect_one()) {
          mbar_expect_tx(&full[st], (uint32_t)(bn * 128));
          tma_load_2d(smem + st * stage_bytes + kABytes, &xmap, (2 * c0 + s) * kStepK, t0, &full[st]);
        }
        __syncwarp();
        if (++st == S) st = 0, par ^= 1;
      }
    }
    // On an error path the producers may stop short of completing a phase:
    // give the copies already issued time to land before the CTA exits.
    if (__any_sync(0xffffffffu, ld_relaxed_i32(p.err) != 0)) {
      const uint64_t w0 = global_timer();
      while (global_timer() - w0 < 200000ull) {
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ MMA issue
    dep_wait();
    dep_release();
    int st = 0, j = 0;
    uint32_t par = 0;
    const uint32_t idesc = idesc_f16_m128(bn);
    for (int u = u0; u < p.units; u += ustep, ++j) {
      const int b = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&tempty[b], ((j >> 1) & 1) ^ 1, p.err, tmo))) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(b * bn);
      bool ok = true;
      for (int s = 0; s < steps; ++s) {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], par, p.err, tmo))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + st * stage_bytes);
        const uint64_t da = smem_desc_sw128(a), db = smem_desc_sw128(a + kABytes);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) umma_f16(d, da + 2 * k, db + 2 * k, idesc, (s | k) ? 1u : 0u);
          umma_commit(&empty[st]);
        }
        __syncwarp();
        if (++st == S) st = 0, par ^= 1;
      }
      if (!ok) break;
      if (elect_one()) umma_commit(&tfull[b]);
      __syncwarp();
    }
    // On an error path, wait (bounded) until the MMAs issued are complete, so
    // that none still writes TMEM when it is released.
    if (__any_sync(0xffffffffu, ld_relaxed_i32(p.err) != 0)) {
      if (elect_one()) umma_commit(tdrain);
      __syncwarp();
      drain_wait(tdrain, 0, tmo);
    }
    __syncwarp();
  }

  if (split > 1) {
    __syncwarp();
    cluster_sync();  // every partial tile is in its CTA's shared memory
    if (warp < 4) {
      const int r = warp * 32 + lane;
      const int row = (u0 % p.n_rb) * kRowsA + r, t0 = (u0 / p.n_rb) * bn;
      const int nt = min(bn, p.T - t0);
      if (row < p.w.N) {
        const float rf = __ldg(p.w.row_f + row) * 0x1p21f;
        const float bias = p.w.bias ? __ldg(p.w.bias + row) : 0.0f;
        const uint32_t part = smem_u32(smem) + 4 * r;
        for (int c = rank; c < nt; c += split) {
          float v = 0.0f;
          for (int k = 0; k < split; ++k) v += ld_cluster_f32(part + c * kRowsA * 4, k);
          const int t = t0 + c;
          p.y[(size_t)t * p.w.N + row] =
              __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(v * rf, p.x_f[t], bias)));
        }
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its tile is read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// Shape of a launch.
struct Plan {
  int bn, units, split, stages, smem, tmem_cols;
};

// Tokens per tile and CTAs per tile, by an estimate of the time in cycles:
// a step of 64 inputs takes 2 cycles per token on the tensor core and about
// 170 in the producers, whichever is longer; 2500 cycles per tile for its
// start and epilogue, 1500 more for the sum over a cluster.
Plan plan(int N, int kc, int T, int num_sms) {
  Plan best = {};
  double best_t = 0.0;
  const int rb = (N + kRowsA - 1) / kRowsA;
  const int j0 = (T + 255) / 256;
  for (int j = j0; j <= j0 + 8; ++j) {
    const int bn = ((T + j - 1) / j + 15) / 16 * 16;
    if (j > j0 && bn < 32) break;
    const int tt = (T + bn - 1) / bn;
    if ((long long)rb * tt > 0x3fffffff) break;
    const int units = rb * tt;
    for (int split = 1; split <= 8 && split <= kc; split *= 2) {
      if (split > 1 && units * split > num_sms) break;
      const int rounds = (units * split + num_sms - 1) / num_sms;
      const double steps = 2.0 * ((kc + split - 1) / split);
      const double t = rounds * (steps * std::max(2 * bn, 170) + 2500) + (split > 1 ? 1500 : 0);
      if (best_t == 0.0 || t < best_t) {
        best_t = t;
        best.bn = bn;
        best.units = units;
        best.split = split;
      }
    }
  }
  const int stage = kABytes + best.bn * 128;
  best.stages = std::min(kMaxStages, (kMaxSmem - 1024 - kRingBytes - kBarBytes) / stage);
  best.smem = best.stages * stage + kRingBytes + kBarBytes + 1024;
  // (S stages always hold the fp32 tile of a shared unit: S >= 3 up to 256
  // tokens, and smaller tiles have at least that ratio)
  best.tmem_cols = 32;
  while (best.tmem_cols < 2 * best.bn) best.tmem_cols *= 2;
  return best;
}
static_assert(3 * (kABytes + 256 * 128) + kRingBytes + kBarBytes + 1024 <= kMaxSmem, "three stages at 256 tokens");
static_assert(3 * (kABytes + 256 * 128) >= 256 * kRowsA * 4, "an fp32 tile fits in the stages");
static_assert(8 * (2 * kMaxStages + 5) + 4 <= kBarBytes, "barriers");

template <bool kQ8>
cudaError_t launch_prep(moe_linear* L, const XIn& in, int T, cudaStream_t s) {
  prof::Scope scope(kQ8 ? "linear_prep_q8" : "linear_prep", s);
  const int nvec = L->w.K / 8;
  __half* x16 = static_cast<__half*>(L->x16);
  if (nvec <= 1024)
    return launch_overlapped(prep_kernel<kQ8, 1>, dim3(T), dim3((nvec + 31) / 32 * 32), 0, s, in, L->w.K, x16, L->x_f);
  return launch_overlapped(prep_kernel<kQ8, 4>, dim3(T), dim3(((nvec + 3) / 4 + 31) / 32 * 32), 0, s, in, L->w.K, x16,
                           L->x_f);
}

}  // namespace

size_t gemm_workspace(int K, int max_tokens) {
  if (max_tokens <= kSmallTokens) return 0;
  return (((size_t)max_tokens * K * 2 + 255) & ~(size_t)255) + (size_t)max_tokens * 4;
}

moe_status gemm_init(moe_linear* L, void* ws) {
  const int T = L->cfg.max_tokens, K = L->w.K;
  if (T <= kSmallTokens) return MOE_OK;
  L->x16 = ws;
  L->x_f = reinterpret_cast<float*>(static_cast<char*>(ws) + (((size_t)T * K * 2 + 255) & ~(size_t)255));
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encode_fn();
  if (!enc) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  for (int i = 0; i < 16; ++i) {
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)T};
    cuuint64_t strides[1] = {(cuuint64_t)K * 2};
    cuuint32_t box[2] = {kStepK, (cuuint32_t)(16 * (i + 1))};
    cuuint32_t es[2] = {1, 1};
    CUresult r = enc(&L->xmap[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, L->x16, dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
  static const cudaError_t attr =
      cudaFuncSetAttribute(gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (attr != cudaSuccess) return cuda_fail(attr, "gemm shared memory");
  return MOE_OK;
}

moe_status launch_gemm(moe_linear* L, const XIn& in, int T, uint16_t* y, cudaStream_t s) {
  cudaError_t e = in.x ? launch_prep<false>(L, in, T, s) : launch_prep<true>(L, in, T, s);
  if (e != cudaSuccess) return cuda_fail(e, "linear prep launch");
  const Plan pl = plan(L->w.N, L->w.kc, T, L->num_sms);
  GemmParams p = {};
  p.w = L->w;
  p.x_f = L->x_f;
  p.y = y;
  p.T = T;
  p.bn = pl.bn;
  p.n_rb = (L->w.N + kRowsA - 1) / kRowsA;
  p.units = pl.units;
  p.split = pl.split;
  p.stages = pl.stages;
  p.tmem_cols = pl.tmem_cols;
  p.err = L->err;
  p.timeout_ns = wait_timeout_ns();
  prof::Scope scope("linear_gemm", s);
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(pl.split > 1 ? pl.units * pl.split : std::min(pl.units, L->num_sms));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = pl.smem;
  c.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = pl.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 2;
  e = cudaLaunchKernelEx(&c, gemm_kernel, p, L->xmap[pl.bn / 16 - 1]);
  if (e != cudaSuccess) return cuda_fail(e, "linear gemm launch");
  return MOE_OK;
}

}  // namespace lin
}  // namespace moe
