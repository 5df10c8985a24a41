// Query and key norms per head with the position rotation in the same pass,
// for the training layout (forward and backward) and for serving, where K and
// V go straight into the paged cache.
//
// For a head row x of width d at position m, with weights w:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = n w,
//   z = R(m) y: the first rd elements in pairs (a, b), turned by the angle of
//   pair f at position m: (a cos - b sin, b cos + a sin). The pairs are
//   (f, f + rd / 2), or (2 f, 2 f + 1) when interleaved; elements from rd on
//   pass through.
// Without weights there is no norm: z = R(m) x.
// Backward, from dz: dy = R(-m) dz, dw = sum over rows of dy n, and with
//   g = dy w: dx = r (g - n mean(g n)).
//
// What bounds them: HBM. Each element is read once and written once (the
// backward reads x and dz), a few FMAs each. So a head row stays in registers
// between its load and its store: d / 8 lanes hold 8 elements (16 bytes) each,
// the mean is a shuffle reduction over them, and a rotation partner half a
// rotated width away is rd / 16 lanes away, another shuffle. A group of lanes
// takes kHeads head rows of one token: their loads are all in flight before
// the first is used, and they share the token's angles.
//
// All arithmetic is in 32 bits; the result is rounded to bf16 once. The weight
// gradients are summed in 32 bits in a fixed order: over a thread's rows, the
// CTA's lanes, then the CTAs' partial sums by a second kernel. No atomics.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kNrThreads = 256;
constexpr int kHeads = 4;  // head rows a group has in flight

struct Angles {
  float c[8], s[8];  // per element; interleaved: s carries the sign too
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// This lane's 8 weights, or nothing.
__device__ __forceinline__ void load_weights(const void* w, int w_bf16, int lane, float (&out)[8]) {
  if (w_bf16) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + lane), out);
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w) + 2 * lane);
    const float4 b = __ldg(reinterpret_cast<const float4*>(w) + 2 * lane + 1);
    out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
    out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
  }
}

// The angles of this lane's 8 elements at position m. Lanes from rd / 8 on hold
// elements that pass through (cos 1, sin 0).
template <bool INTER>
__device__ __forceinline__ void load_angles(const float* cos_t, const float* sin_t, long long m, int rd, int lane,
                                            Angles& a) {
  const int half_lanes = rd / 16;
  if (8 * lane >= rd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a.c[e] = 1.f, a.s[e] = 0.f;
    return;
  }
  if (INTER) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cos_t + m * (rd / 2)) + lane);
    const float4 s = __ldg(reinterpret_cast<const float4*>(sin_t + m * (rd / 2)) + lane);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a.c[2 * i] = a.c[2 * i + 1] = cc[i];
      a.s[2 * i] = -ss[i];
      a.s[2 * i + 1] = ss[i];
    }
  } else {
    const bool upper = lane >= half_lanes;
    const int f = 2 * (lane - (upper ? half_lanes : 0));
    const float4* cp = reinterpret_cast<const float4*>(cos_t + m * (rd / 2)) + f;
    const float4* sp = reinterpret_cast<const float4*>(sin_t + m * (rd / 2)) + f;
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    const float sg = upper ? 1.f : -1.f;
    a.c[0] = c0.x, a.c[1] = c0.y, a.c[2] = c0.z, a.c[3] = c0.w;
    a.c[4] = c1.x, a.c[5] = c1.y, a.c[6] = c1.z, a.c[7] = c1.w;
    a.s[0] = sg * s0.x, a.s[1] = sg * s0.y, a.s[2] = sg * s0.z, a.s[3] = sg * s0.w;
    a.s[4] = sg * s1.x, a.s[5] = sg * s1.y, a.s[6] = sg * s1.z, a.s[7] = sg * s1.w;
  }
}

// y turned by the angles (dir = 1) or back (dir = -1). `partner`: the warp lane
// that holds the other half of this lane's pairs.
// Elements that pass through are left alone (an infinity times sin 0 is NaN).
template <bool INTER>
__device__ __forceinline__ void rotate8(float (&y)[8], const Angles& a, float dir, int partner, bool turned) {
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = INTER ? y[e ^ 1] : __shfl_sync(0xffffffffu, y[e], partner);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = turned ? fmaf(o[e], dir * a.s[e], y[e] * a.c[e]) : y[e];
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int s = LANES / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

struct HeadView {  // [.., token, head, d] bf16, strides in elements
  const __nv_bfloat16* p;
  long long sb, sn, sh;
};

struct NormRopeParams {
  HeadView in[3];  // q, k, v
  const void* w[2];
  const float* cos_t;
  const float* sin_t;
  const int32_t* positions;  // null: the token's index in its sequence
  const int32_t* slots;      // paged only
  __nv_bfloat16* out[3];     // dense: [B, H, N, d] each; paged: q [T, Hq, d] and the two pools
  int32_t* status;
  unsigned tokens;  // B * N, or T; tokens * chunks < 2^31
  int N, Hq, Hkv, rd, max_pos, chunks, w_bf16;
  long long num_slots;
  float eps;
};

// Which tensor (0 q, 1 k, 2 v) and which of its heads is head h of a token.
__device__ __forceinline__ int tensor_of(int& h, int Hq, int Hkv) {
  if (h < Hq) return 0;
  h -= Hq;
  if (h < Hkv) return 1;
  h -= Hkv;
  return 2;
}

template <int D, bool INTER, bool NORM, bool PAGED>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kNrThreads / kLanes;
  const int lane = threadIdx.x & (kLanes - 1);
  const unsigned unit = blockIdx.x * kGroups + threadIdx.x / kLanes;
  const unsigned units = p.tokens * p.chunks;
  const unsigned tok = unit < units ? unit / p.chunks : p.tokens - 1;  // every lane stays for the shuffles
  const int h0 = unit < units ? (unit - tok * p.chunks) * kHeads : 0;
  const long long token = tok, b = PAGED ? 0 : tok / p.N;
  const int n = static_cast<int>(token - b * p.N);
  const int heads = p.Hq + 2 * p.Hkv;

  uint4 raw[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    int h = h0 + i;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (h < heads) {
      const int t = tensor_of(h, p.Hq, p.Hkv);
      const HeadView& v = p.in[t];
      const long long row = PAGED ? token * v.sn : b * v.sb + static_cast<long long>(n) * v.sn;
      raw[i] = __ldg(reinterpret_cast<const uint4*>(v.p + row + h * v.sh) + lane);
    }
  }
  const long long m = p.positions != nullptr ? __ldg(p.positions + token) : n;
  const bool bad = m < 0 || m >= p.max_pos;
  Angles a;
  load_angles<INTER>(p.cos_t, p.sin_t, bad ? 0 : m, p.rd, lane, a);
  long long slot = -1;
  bool bad_slot = false;
  if (PAGED && h0 + kHeads > p.Hq) {
    slot = __ldg(p.slots + token);
    bad_slot = slot < -1 || slot >= p.num_slots;
  }
  const int half_lanes = p.rd / 16;
  const bool turned = 8 * lane < p.rd;
  const int partner = (threadIdx.x & 31) + (!turned ? 0 : (lane >= half_lanes ? -half_lanes : half_lanes));

#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    int h = h0 + i;
    const bool there = unit < units && h < heads;
    const int t = tensor_of(h, p.Hq, p.Hkv);
    uint4 res = raw[i];
    // a warp's groups may hold heads of different tensors: the shuffles run for all
    float y[8];
    unpack8(raw[i], y);
    if (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
      const float r = rsqrtf(group_sum<kLanes>(ss) * (1.f / D) + p.eps);
      float w[8];
      load_weights(p.w[t == 1 ? 1 : 0], p.w_bf16, lane, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= r * w[e];
    }
    rotate8<INTER>(y, a, 1.f, partner, turned);
    if (t < 2) {
      if (bad) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = NAN;
      }
      res = pack8(y);
    }
    if (!there) continue;
    __nv_bfloat16* dst;
    if (!PAGED) {
      const int H = t == 0 ? p.Hq : p.Hkv;
      dst = p.out[t] + ((b * H + h) * p.N + n) * D;
    } else if (t == 0) {
      dst = p.out[0] + (token * p.Hq + h) * D;
    } else {
      if (slot < 0 || bad_slot || bad) continue;
      dst = p.out[t] + (slot * p.Hkv + h) * D;
    }
    reinterpret_cast<uint4*>(dst)[lane] = res;
  }
  if ((bad || bad_slot) && unit < units && lane == 0 && p.status != nullptr)
    atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
}

struct NormRopeBwdParams {
  HeadView x[2];             // q, k (unused without norms)
  const void* w[2];
  const float* cos_t;
  const float* sin_t;
  const int32_t* positions;
  const __nv_bfloat16* dz[3];  // [B, H, N, d]
  __nv_bfloat16* dx[3];        // strided like the inputs
  long long dsb[3], dsn[3], dsh[3];
  float* dw_part;  // [ctas, 2, d]
  int32_t* status;
  unsigned tokens;
  int N, Hq, Hkv, rd, max_pos, chunks, w_bf16;
  float eps;
};

template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kNrThreads) norm_rope_bwd_kernel(const NormRopeBwdParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kNrThreads / kLanes;
  __shared__ float dw_s[kNrThreads / 32][2][D];
  const int lane = threadIdx.x & (kLanes - 1);
  const unsigned units = p.tokens * p.chunks;
  const int heads = p.Hq + 2 * p.Hkv;
  const int half_lanes = p.rd / 16;
  const bool turned = 8 * lane < p.rd;
  const int partner = (threadIdx.x & 31) + (!turned ? 0 : (lane >= half_lanes ? -half_lanes : half_lanes));
  float dwq[8], dwk[8], wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = wq[e] = wk[e] = 0.f;
  if (NORM) {
    load_weights(p.w[0], p.w_bf16, lane, wq);
    load_weights(p.w[1], p.w_bf16, lane, wk);
  }
  bool any_bad = false;
  for (unsigned base = blockIdx.x * kGroups; base < units; base += gridDim.x * kGroups) {
    const unsigned unit = base + threadIdx.x / kLanes;
    const bool live = unit < units;
    const unsigned tok = live ? unit / p.chunks : p.tokens - 1;
    const int h0 = live ? (unit - tok * p.chunks) * kHeads : 0;
    const long long token = tok, b = tok / p.N;
    const int n = static_cast<int>(token - b * p.N);
    uint4 rx[kHeads], rz[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      int h = h0 + i;
      rx[i] = rz[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h < heads) {
        const int t = tensor_of(h, p.Hq, p.Hkv);
        const int H = t == 0 ? p.Hq : p.Hkv;
        rz[i] = __ldg(reinterpret_cast<const uint4*>(p.dz[t] + ((b * H + h) * p.N + n) * D) + lane);
        if (NORM && t < 2)
          rx[i] = __ldg(reinterpret_cast<const uint4*>(p.x[t].p + b * p.x[t].sb + static_cast<long long>(n) * p.x[t].sn +
                                                       h * p.x[t].sh) + lane);
      }
    }
    const long long m = p.positions != nullptr ? __ldg(p.positions + token) : n;
    const bool bad = m < 0 || m >= p.max_pos;
    any_bad |= bad && live;
    Angles a;
    load_angles<INTER>(p.cos_t, p.sin_t, bad ? 0 : m, p.rd, lane, a);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      int h = h0 + i;
      const bool there = live && h < heads;
      const int t = tensor_of(h, p.Hq, p.Hkv);
      float g[8];
      unpack8(rz[i], g);
      rotate8<INTER>(g, a, -1.f, partner, turned);
      if (bad) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = NAN;
      }
      if (NORM) {
        float x[8];
        unpack8(rx[i], x);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(group_sum<kLanes>(ss) * (1.f / D) + p.eps);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= r;  // n
          const float d = g[e] * x[e];
          if (there && t == 0) dwq[e] += d;
          if (there && t == 1) dwk[e] += d;
          const float w = t == 1 ? wk[e] : wq[e];
          dot = fmaf(d, w, dot);
          g[e] *= w;
        }
        dot = group_sum<kLanes>(dot) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-x[e], dot, g[e]);
      }
      if (!there) continue;
      const uint4 res = t < 2 ? pack8(g) : rz[i];
      __nv_bfloat16* dst = p.dx[t] + b * p.dsb[t] + static_cast<long long>(n) * p.dsn[t] + h * p.dsh[t];
      reinterpret_cast<uint4*>(dst)[lane] = res;
    }
  }
  if (any_bad && lane == 0 && p.status != nullptr) atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
  if (NORM) {
    // lanes with the same elements: the warp's groups, then the CTA's warps, in that order
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int s = kLanes; s < 32; s <<= 1) {
        dwq[e] += __shfl_xor_sync(0xffffffffu, dwq[e], s);
        dwk[e] += __shfl_xor_sync(0xffffffffu, dwk[e], s);
      }
      if ((threadIdx.x & 31) < kLanes) {
        dw_s[threadIdx.x >> 5][0][8 * lane + e] = dwq[e];
        dw_s[threadIdx.x >> 5][1][8 * lane + e] = dwk[e];
      }
    }
    __syncthreads();
    if (threadIdx.x < 2 * D) {
      float s = 0.f;
#pragma unroll
      for (int wp = 0; wp < kNrThreads / 32; ++wp) s += (&dw_s[wp][0][0])[threadIdx.x];
      p.dw_part[static_cast<long long>(blockIdx.x) * 2 * D + threadIdx.x] = s;
    }
  }
}

// dw = sum over the CTAs' partial rows: a CTA takes 32 columns, its 32 warps
// every 32nd row each, then one warp adds the 32 sums.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int rows, float* dwq, float* dwk) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
  for (int r = warp; r < rows; r += 32) v += part[static_cast<long long>(r) * 2 * D + col];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][lane];
    (col < D ? dwq : dwk)[col < D ? col : col - D] = t;
  }
}

template <int D, bool INTER, bool NORM, bool PAGED>
int launch_fwd_t(const NormRopeParams& p, cudaStream_t stream) {
  const long long groups = kNrThreads / (D / 8);
  const long long blocks = (static_cast<long long>(p.tokens) * p.chunks + groups - 1) / groups;
  norm_rope_kernel<D, INTER, NORM, PAGED><<<static_cast<unsigned>(blocks), kNrThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
template <bool PAGED>
int launch_fwd(const NormRopeParams& p, int d, int interleaved, cudaStream_t stream) {
  const bool norm = p.w[0] != nullptr;
  if (d == 128)
    return interleaved ? (norm ? launch_fwd_t<128, true, true, PAGED>(p, stream)
                               : launch_fwd_t<128, true, false, PAGED>(p, stream))
                       : (norm ? launch_fwd_t<128, false, true, PAGED>(p, stream)
                               : launch_fwd_t<128, false, false, PAGED>(p, stream));
  return interleaved ? (norm ? launch_fwd_t<64, true, true, PAGED>(p, stream)
                             : launch_fwd_t<64, true, false, PAGED>(p, stream))
                     : (norm ? launch_fwd_t<64, false, true, PAGED>(p, stream)
                             : launch_fwd_t<64, false, false, PAGED>(p, stream));
}

template <int D, bool INTER, bool NORM>
int launch_bwd_t(const NormRopeBwdParams& p, int ctas, float* dwq, float* dwk, cudaStream_t stream) {
  norm_rope_bwd_kernel<D, INTER, NORM><<<ctas, kNrThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (!NORM) return ATTN_OK;
  norm_rope_dw_kernel<D><<<2 * D / 32, 1024, 0, stream>>>(p.dw_part, ctas, dwq, dwk);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

int norm_rope_chunks(int Hq, int Hkv) { return (Hq + 2 * Hkv + kHeads - 1) / kHeads; }

int norm_rope_bwd_ctas(long long tokens, int Hq, int Hkv, int d, int sms) {
  const long long groups = kNrThreads / (d / 8);
  const long long blocks = (tokens * norm_rope_chunks(Hq, Hkv) + groups - 1) / groups;
  const long long most = 4LL * sms;
  return static_cast<int>(blocks < most ? blocks : most);
}

int launch_norm_rope(const NormRopeArgs& a, void* q_out, void* k_out, void* v_out, const int32_t* slots,
                     long long num_slots, int32_t* status, cudaStream_t stream) {
  NormRopeParams p{};
  for (int t = 0; t < 3; ++t)
    p.in[t] = HeadView{static_cast<const __nv_bfloat16*>(a.x[t]), a.sb[t], a.sn[t], a.sh[t]};
  p.w[0] = a.w[0];
  p.w[1] = a.w[1];
  p.cos_t = a.cos_t;
  p.sin_t = a.sin_t;
  p.positions = a.positions;
  p.slots = slots;
  p.out[0] = static_cast<__nv_bfloat16*>(q_out);
  p.out[1] = static_cast<__nv_bfloat16*>(k_out);
  p.out[2] = static_cast<__nv_bfloat16*>(v_out);
  p.status = status;
  p.tokens = static_cast<unsigned>(a.B) * a.N;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.rd = a.rd;
  p.max_pos = a.max_pos;
  p.chunks = norm_rope_chunks(a.Hq, a.Hkv);
  p.w_bf16 = a.w_bf16;
  p.num_slots = num_slots;
  p.eps = a.eps;
  return slots != nullptr ? launch_fwd<true>(p, a.d, a.interleaved, stream)
                          : launch_fwd<false>(p, a.d, a.interleaved, stream);
}

int launch_norm_rope_backward(const NormRopeArgs& a, const void* const dz[3], void* const dx[3], const int64_t dsb[3],
                              const int64_t dsn[3], const int64_t dsh[3], float* dwq, float* dwk, float* dw_part,
                              int ctas, int32_t* status, cudaStream_t stream) {
  NormRopeBwdParams p{};
  for (int t = 0; t < 2; ++t)
    p.x[t] = HeadView{static_cast<const __nv_bfloat16*>(a.x[t]), a.sb[t], a.sn[t], a.sh[t]};
  for (int t = 0; t < 3; ++t) {
    p.dz[t] = static_cast<const __nv_bfloat16*>(dz[t]);
    p.dx[t] = static_cast<__nv_bfloat16*>(dx[t]);
    p.dsb[t] = dsb[t];
    p.dsn[t] = dsn[t];
    p.dsh[t] = dsh[t];
  }
  p.w[0] = a.w[0];
  p.w[1] = a.w[1];
  p.cos_t = a.cos_t;
  p.sin_t = a.sin_t;
  p.positions = a.positions;
  p.dw_part = dw_part;
  p.status = status;
  p.tokens = static_cast<unsigned>(a.B) * a.N;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.rd = a.rd;
  p.max_pos = a.max_pos;
  p.chunks = norm_rope_chunks(a.Hq, a.Hkv);
  p.w_bf16 = a.w_bf16;
  p.eps = a.eps;
  const bool norm = a.w[0] != nullptr;
  if (a.d == 128)
    return a.interleaved ? (norm ? launch_bwd_t<128, true, true>(p, ctas, dwq, dwk, stream)
                                 : launch_bwd_t<128, true, false>(p, ctas, dwq, dwk, stream))
                         : (norm ? launch_bwd_t<128, false, true>(p, ctas, dwq, dwk, stream)
                                 : launch_bwd_t<128, false, false>(p, ctas, dwq, dwk, stream));
  return a.interleaved ? (norm ? launch_bwd_t<64, true, true>(p, ctas, dwq, dwk, stream)
                               : launch_bwd_t<64, true, false>(p, ctas, dwq, dwk, stream))
                       : (norm ? launch_bwd_t<64, false, true>(p, ctas, dwq, dwk, stream)
                               : launch_bwd_t<64, false, false>(p, ctas, dwq, dwk, stream));
}

}  // namespace attn
