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
// rotated width away is rd / 16 lanes away: its raw 16 bytes come by 4 shuffles.
// At a full HBM's pace an SM has 44 cycles for a warp's 512 bytes, so the
// instructions count too: pairs of elements share one (f32x2), and weights and
// angles are multiplied once a token, not once a head.
//
// A group of lanes takes one token, and kHeads heads of one tensor at a time,
// copied to shared memory one step ahead. The groups of a CTA take the same heads
// of consecutive tokens: a head's rows then lie together on the [B, H, N, d] side
// (4 KB at d = 128), a token's heads on the other (1 KB), and angles and weights
// are read once for all heads of the CTA. Measured for B = 4, N = 4096, 32 / 8
// heads, d = 128 (forward 405 MB, backward 573 MB), all forms in turn on one card,
// three sets of inputs in turn, medians: one group per 4 heads of a token, groups on
// a token's heads 117 and 168 us; groups on consecutive tokens 85 and 131; all heads
// of a token in turn 76 and 127; the steps prefetched 69 (89 % of HBM) and 116; the
// backward's two sums a row taken side by side 112, its CTAs' shares even in rows
// moved 100 (87 %; a third CTA an SM, at 80 registers, takes 112, a third step in the
// ring 106).
//
// All arithmetic is in 32 bits; the result is rounded to bf16 once. The weight
// gradients are summed in 32 bits in a fixed order: the 4 rows of a step, a
// thread's steps one after another, the CTA's lanes, then the CTAs' partial sums by
// a second kernel. No atomics. So their rounding is at most 2^-24 of the sum of
// |dy n| for each of a thread's steps (42 for the training shapes above, in
// proportion to tokens and heads beyond one wave of CTAs) and for each of some 60
// additions after them.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kNrThreads = 256;
constexpr int kHeads = 4;  // head rows a group has in flight
constexpr int kFwdCtasPerSm = 8;
constexpr int kBwdCtasPerSm = 2;

using F2x4 = float2[4];  // a lane's 8 elements

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void unpack8(const uint4& v, F2x4& x) {
  x[0] = unpack2(v.x), x[1] = unpack2(v.y), x[2] = unpack2(v.z), x[3] = unpack2(v.w);
}
__device__ __forceinline__ uint4 pack8(const F2x4& x) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                    pack_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ float2 swap2(float2 v) { return make_float2(v.y, v.x); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// This lane's 8 weights.
__device__ __forceinline__ void load_weights(const void* w, int w_bf16, int lane, F2x4& out) {
  if (w_bf16) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + lane), out);
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w) + 2 * lane);
    const float4 b = __ldg(reinterpret_cast<const float4*>(w) + 2 * lane + 1);
    out[0] = make_float2(a.x, a.y), out[1] = make_float2(a.z, a.w);
    out[2] = make_float2(b.x, b.y), out[3] = make_float2(b.z, b.w);
  }
}

// What the elements of a lane are multiplied with at position m: own element by
// c, partner's by s (the sign of the rotation included; dir = -1 turns back).
// Lanes from rd / 8 on hold elements that pass through: c = 1, s = 0, and a
// partner of 0 (an infinity times 0 would be NaN).
template <bool INTER>
__device__ __forceinline__ void load_angles(const float* cos_t, const float* sin_t, long long m, int rd, int lane,
                                            float dir, F2x4& c, F2x4& s) {
  if (8 * lane >= rd) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = both(1.f), s[i] = both(0.f);
    return;
  }
  if (INTER) {
    const float4 cv = __ldg(reinterpret_cast<const float4*>(cos_t + m * (rd / 2)) + lane);
    const float4 sv = __ldg(reinterpret_cast<const float4*>(sin_t + m * (rd / 2)) + lane);
    const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = both(cc[i]), s[i] = make_float2(-dir * ss[i], dir * ss[i]);
  } else {
    const bool upper = lane >= rd / 16;
    const int f = 2 * (lane - (upper ? rd / 16 : 0));
    const float4* cp = reinterpret_cast<const float4*>(cos_t + m * (rd / 2)) + f;
    const float4* sp = reinterpret_cast<const float4*>(sin_t + m * (rd / 2)) + f;
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    const float sg = upper ? dir : -dir;
    c[0] = make_float2(c0.x, c0.y), c[1] = make_float2(c0.z, c0.w);
    c[2] = make_float2(c1.x, c1.y), c[3] = make_float2(c1.z, c1.w);
    s[0] = make_float2(sg * s0.x, sg * s0.y), s[1] = make_float2(sg * s0.z, sg * s0.w);
    s[2] = make_float2(sg * s1.x, sg * s1.y), s[3] = make_float2(sg * s1.z, sg * s1.w);
  }
}

// The partners of a lane's elements. `partner`: the warp lane that holds them.
template <bool INTER>
__device__ __forceinline__ void partner8(const uint4& raw, const F2x4& x, int partner, bool turned, F2x4& out) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = turned ? swap2(x[i]) : both(0.f);
    return;
  }
  uint4 o;
  o.x = __shfl_sync(0xffffffffu, raw.x, partner);
  o.y = __shfl_sync(0xffffffffu, raw.y, partner);
  o.z = __shfl_sync(0xffffffffu, raw.z, partner);
  o.w = __shfl_sync(0xffffffffu, raw.w, partner);
  if (!turned) o = make_uint4(0u, 0u, 0u, 0u);
  unpack8(o, out);
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int s = LANES / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}
__device__ __forceinline__ float dot8(const F2x4& a, const F2x4& b) {
  float2 v = fmul2(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) v = ffma2(a[i], b[i], v);
  return v.x + v.y;
}

// A thread's own ring of 16-byte pieces in shared memory: cp.async fills a step's
// pieces kSteps - 1 steps ahead, the same thread reads them, so the loads in flight
// cost no registers and no barrier. A step's pieces are written over those of the
// step before the current one, whose values are long used.
constexpr int kSteps = 2;
template <int PIECES>
struct Ring {
  static constexpr int kBytes = kSteps * PIECES * kNrThreads * 16;
  uint32_t base;
  const uint4* mem;
  __device__ __forceinline__ explicit Ring(uint4* smem) : base(smem_u32(smem + threadIdx.x)), mem(smem + threadIdx.x) {}
  __device__ __forceinline__ void load(int slot, int i, const void* src) {
    cp_async_16(base + (slot * PIECES + i) * kNrThreads * 16, src, 16);
  }
  __device__ __forceinline__ uint4 get(int slot, int i) const { return mem[(slot * PIECES + i) * kNrThreads]; }
};
__device__ __forceinline__ int next_slot(int slot) { return slot + 1 == kSteps ? 0 : slot + 1; }

struct HeadView {  // [.., token, head, d] bf16, strides in elements
  const __nv_bfloat16* p;
  long long sb, sn, sh;
};

// The heads of the three tensors in chunks of kHeads that do not cross tensors.
struct Chunks {
  int q, kv;  // chunks of q, of k and of v each
  __host__ __device__ int all() const { return q + 2 * kv; }
};
__host__ __device__ inline Chunks chunks_of(int Hq, int Hkv) {
  return Chunks{(Hq + kHeads - 1) / kHeads, (Hkv + kHeads - 1) / kHeads};
}
struct HeadRange {
  int t, h0, cnt;  // tensor (0 q, 1 k, 2 v), first head, heads
};
__device__ __forceinline__ HeadRange heads_of(const Chunks& ch, int chunk, int Hq, int Hkv) {
  const int t = chunk < ch.q ? 0 : (chunk < ch.q + ch.kv ? 1 : 2);
  const int h0 = (chunk - (t == 0 ? 0 : ch.q + (t - 1) * ch.kv)) * kHeads;
  return HeadRange{t, h0, min(kHeads, (t == 0 ? Hq : Hkv) - h0)};
}

struct NormRopeParams {
  HeadView in[3];  // q, k, v
  const void* w[2];
  const float* cos_t;
  const float* sin_t;
  const int32_t* positions;  // null: the token's index in its sequence
  const int32_t* slots;      // paged only
  __nv_bfloat16* out[3];     // dense: [B, H, N, d] each; paged: q [T, Hq, d] and the two pools
  int32_t* status;
  unsigned tokens;  // B * N, or T
  int N, Hq, Hkv, rd, max_pos, w_bf16, parts;
  Chunks ch;
  long long num_slots;
  float eps;
};

// CTA blockIdx.x: a tile of tokens, and of the chunks the part [all part / parts, all (part + 1) / parts).
template <int D, bool INTER, bool NORM, bool PAGED>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kNrThreads / kLanes;
  const int lane = threadIdx.x & (kLanes - 1);
  const unsigned tile = blockIdx.x / p.parts;
  const int part = static_cast<int>(blockIdx.x - tile * p.parts), all = p.ch.all();
  const int c_begin = all * part / p.parts, c_end = all * (part + 1) / p.parts;
  const unsigned at = tile * kGroups + threadIdx.x / kLanes;
  const bool live = at < p.tokens;
  const unsigned tok = live ? at : p.tokens - 1;  // every lane stays for the shuffles
  const long long token = tok, b = PAGED ? 0 : tok / p.N;
  const int n = static_cast<int>(token - b * p.N);
  extern __shared__ uint4 ring_smem[];
  Ring<kHeads> ring(ring_smem);
  int slot_at = 0, slot_in = 0;
  auto fetch = [&](int chunk) {
    if (chunk < c_end) {
      const HeadRange hr = heads_of(p.ch, chunk, p.Hq, p.Hkv);
      const HeadView& v = p.in[hr.t];
      const __nv_bfloat16* src =
          v.p + b * v.sb + static_cast<long long>(PAGED ? tok : n) * v.sn + hr.h0 * v.sh + 8 * lane;
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
        if (i < hr.cnt) ring.load(slot_in, i, src + i * v.sh);
      slot_in = next_slot(slot_in);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kSteps - 1; ++i) fetch(c_begin + i);
  const long long m = p.positions != nullptr ? __ldg(p.positions + token) : n;
  const bool bad = m < 0 || m >= p.max_pos;
  long long slot = -1;
  bool bad_slot = false;
  if (PAGED) {
    slot = __ldg(p.slots + token);
    bad_slot = slot < -1 || slot >= p.num_slots;
    if (bad_slot || bad) slot = -1;
  }
  if ((bad || bad_slot) && live && lane == 0 && p.status != nullptr)
    atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
  const int half_lanes = p.rd / 16;
  const bool turned = 8 * lane < p.rd;
  const int shift = !turned ? 0 : (lane >= half_lanes ? -half_lanes : half_lanes);
  const int partner = (threadIdx.x & 31) + shift;
  F2x4 c, s;
  int loaded = -1;  // the tensor whose weights c and s hold

  for (int chunk = c_begin; chunk < c_end; ++chunk, slot_at = next_slot(slot_at)) {
    const HeadRange hr = heads_of(p.ch, chunk, p.Hq, p.Hkv);
    cp_async_wait<kSteps - 2>();
    fetch(chunk + kSteps - 1);
    bool write = live;
    __nv_bfloat16* dst;
    long long step;  // between heads
    if (!PAGED) {
      const int H = hr.t == 0 ? p.Hq : p.Hkv;
      dst = p.out[hr.t] + ((b * H + hr.h0) * p.N + n) * D;
      step = static_cast<long long>(p.N) * D;
    } else {
      step = D;
      if (hr.t == 0) {
        dst = p.out[0] + (token * p.Hq + hr.h0) * D;
      } else {
        write = live && slot >= 0;
        dst = p.out[hr.t] + ((write ? slot : 0) * p.Hkv + hr.h0) * D;
      }
    }
    if (hr.t == 2) {  // V is carried over
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
        if (write && i < hr.cnt) reinterpret_cast<uint4*>(dst + i * step)[lane] = ring.get(slot_at, i);
      continue;
    }
    if (loaded < 0 || (NORM && loaded != hr.t)) {
      loaded = hr.t;
      load_angles<INTER>(p.cos_t, p.sin_t, bad ? 0 : m, p.rd, lane, 1.f, c, s);
      if (NORM) {  // z = r (x (w c) + partner (its w s))
        F2x4 w, wp;
        load_weights(p.w[hr.t], p.w_bf16, lane, w);
        if (!INTER) load_weights(p.w[hr.t], p.w_bf16, lane + shift, wp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[i] = fmul2(c[i], w[i]);
          s[i] = fmul2(s[i], INTER ? swap2(w[i]) : wp[i]);
        }
      }
      if (bad) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = both(NAN);
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (i >= hr.cnt) break;  // the same for the whole CTA
      const uint4 raw = ring.get(slot_at, i);
      F2x4 x, xp;
      unpack8(raw, x);
      partner8<INTER>(raw, x, partner, turned, xp);
      float2 r = both(1.f);
      if (NORM) r = both(rsqrtf(group_sum<kLanes>(dot8(x, x)) * (1.f / D) + p.eps));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = ffma2(xp[e], s[e], fmul2(x[e], c[e]));
        if (NORM) x[e] = fmul2(x[e], r);
      }
      if (write) reinterpret_cast<uint4*>(dst + i * step)[lane] = pack8(x);
    }
  }
}

struct NormRopeBwdParams {
  HeadView x[2];  // q, k (unused without norms)
  const void* w[2];
  const float* cos_t;
  const float* sin_t;
  const int32_t* positions;
  const __nv_bfloat16* dz[3];  // [B, H, N, d]
  __nv_bfloat16* dx[3];        // strided like the inputs
  long long dsb[3], dsn[3], dsh[3];
  float* dw_part;  // a row of d for each CTA and weight: [2][gridDim.x][d]
  int32_t* status;
  unsigned tokens, tiles;
  int N, Hq, Hkv, rd, max_pos, w_bf16;
  Chunks ch;
  float eps;
};

// The steps (a chunk of a tile of tokens, tile after tile) as a line of tensor
// rows to move: dz, x and dx for a chunk of q or k, dz and dx for one of v or
// without norms. Place `at` on it, rounded up to a step.
struct Step {
  unsigned tile;
  int chunk;
};
template <bool NORM>
__device__ __forceinline__ Step step_at(unsigned long long at, const Chunks& ch) {
  constexpr int kTurned = NORM ? 3 : 2;
  const int turned = ch.q + ch.kv, width = kTurned * turned + 2 * ch.kv;
  Step s;
  s.tile = static_cast<unsigned>(at / width);
  const int in = static_cast<int>(at - static_cast<unsigned long long>(s.tile) * width);
  s.chunk = in <= kTurned * turned ? (in + kTurned - 1) / kTurned : turned + (in - kTurned * turned + 1) / 2;
  if (s.chunk == ch.all()) ++s.tile, s.chunk = 0;
  return s;
}

// CTA blockIdx.x: its share of the line. Two CTAs an SM (figures at the file's
// head). A share ends where it ends: whole tiles for each part of the heads left some
// CTAs with the norms and others with the copies.
template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kNrThreads, kBwdCtasPerSm) norm_rope_bwd_kernel(const NormRopeBwdParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kNrThreads / kLanes;
  __shared__ float dw_s[kNrThreads / 32][D];
  const int lane = threadIdx.x & (kLanes - 1);
  const int all = p.ch.all();
  const unsigned long long line =
      static_cast<unsigned long long>(p.tiles) * ((NORM ? 3 : 2) * (p.ch.q + p.ch.kv) + 2 * p.ch.kv);
  const Step begin = step_at<NORM>(line * blockIdx.x / gridDim.x, p.ch);
  const Step end = step_at<NORM>(line * (blockIdx.x + 1) / gridDim.x, p.ch);
  const int half_lanes = p.rd / 16;
  const bool turned = 8 * lane < p.rd;
  const int partner = (threadIdx.x & 31) + (!turned ? 0 : (lane >= half_lanes ? -half_lanes : half_lanes));
  F2x4 dwq, dwk;
#pragma unroll
  for (int i = 0; i < 4; ++i) dwq[i] = dwk[i] = both(0.f);
  bool any_bad = false;
  struct Place {  // this thread's token of a tile
    bool live;
    unsigned tok;
    long long b;
    int n;
  };
  auto place = [&](unsigned tile) {
    const unsigned at = tile * kGroups + threadIdx.x / kLanes;
    Place w;
    w.live = at < p.tokens;
    w.tok = w.live ? at : p.tokens - 1;
    w.b = w.tok / p.N;
    w.n = static_cast<int>(w.tok - w.b * p.N);
    return w;
  };
  // the summing grid may be set up now; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  extern __shared__ uint4 ring_smem[];
  Ring<2 * kHeads> ring(ring_smem);  // dz's pieces, then x's
  int slot_at = 0, slot_in = 0;
  // the step to fetch next: a chunk of a tile
  Step f = begin;
  Place fp = place(begin.tile);
  auto fetch = [&]() {
    if (f.tile < end.tile || (f.tile == end.tile && f.chunk < end.chunk)) {
      const HeadRange hr = heads_of(p.ch, f.chunk, p.Hq, p.Hkv);
      const __nv_bfloat16* zs =
          p.dz[hr.t] + ((fp.b * (hr.t == 0 ? p.Hq : p.Hkv) + hr.h0) * p.N + fp.n) * D + 8 * lane;
      const long long zstep = static_cast<long long>(p.N) * D;
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
        if (i < hr.cnt) ring.load(slot_in, i, zs + i * zstep);
      if (NORM && hr.t < 2) {
        const HeadView& v = p.x[hr.t];
        const __nv_bfloat16* xs = v.p + fp.b * v.sb + static_cast<long long>(fp.n) * v.sn + hr.h0 * v.sh + 8 * lane;
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
          if (i < hr.cnt) ring.load(slot_in, kHeads + i, xs + i * v.sh);
      }
      slot_in = next_slot(slot_in);
      if (++f.chunk == all) {
        f.chunk = 0;
        fp = place(++f.tile);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kSteps - 1; ++i) fetch();
  for (unsigned tile = begin.tile; tile <= end.tile; ++tile) {
    const int c_begin = tile == begin.tile ? begin.chunk : 0, c_end = tile == end.tile ? end.chunk : all;
    if (c_begin >= c_end) break;  // the share ends with the tile before
    const Place pl = place(tile);
    const bool live = pl.live;
    const unsigned tok = pl.tok;
    const long long b = pl.b;
    const int n = pl.n;
    const long long m = p.positions != nullptr ? __ldg(p.positions + tok) : n;
    const bool bad = m < 0 || m >= p.max_pos;
    any_bad |= bad && live;
    F2x4 c, s;
    load_angles<INTER>(p.cos_t, p.sin_t, bad ? 0 : m, p.rd, lane, -1.f, c, s);
    if (bad) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = both(NAN);
    }
    for (int chunk = c_begin; chunk < c_end; ++chunk, slot_at = next_slot(slot_at)) {
      const HeadRange hr = heads_of(p.ch, chunk, p.Hq, p.Hkv);
      const bool copy = hr.t == 2;
      cp_async_wait<kSteps - 2>();
      fetch();
      __nv_bfloat16* dst =
          p.dx[hr.t] + b * p.dsb[hr.t] + static_cast<long long>(n) * p.dsn[hr.t] + hr.h0 * p.dsh[hr.t];
      const long long step = p.dsh[hr.t];
      if (copy) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
          if (live && i < hr.cnt) reinterpret_cast<uint4*>(dst + i * step)[lane] = ring.get(slot_at, i);
        continue;
      }
      F2x4 w, dw;
      if (NORM) load_weights(p.w[hr.t], p.w_bf16, lane, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) dw[i] = both(0.f);
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        if (i >= hr.cnt) break;
        const uint4 rz = ring.get(slot_at, i);
        F2x4 g, gp;
        unpack8(rz, g);
        partner8<INTER>(rz, g, partner, turned, gp);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = ffma2(gp[e], s[e], fmul2(g[e], c[e]));
        if (NORM) {
          F2x4 x, gw;
          unpack8(ring.get(slot_at, kHeads + i), x);
#pragma unroll
          for (int e = 0; e < 4; ++e) gw[e] = fmul2(g[e], w[e]);
          // sum(g x) r in place of sum(g n): the two sums do not wait for each other
          const float ss = group_sum<kLanes>(dot8(x, x)), gx = group_sum<kLanes>(dot8(gw, x));
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const float t = -(gx * r) * (1.f / D) * r;  // n mean(g n) = -t x
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dw[e] = ffma2(fmul2(g[e], both(r)), x[e], dw[e]);
            g[e] = fmul2(ffma2(x[e], both(t), gw[e]), both(r));
          }
        }
        if (live) reinterpret_cast<uint4*>(dst + i * step)[lane] = pack8(g);
      }
      if (NORM && live) {
        F2x4& sum = hr.t == 0 ? dwq : dwk;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = fadd2(sum[e], dw[e]);
      }
    }
  }
  if (any_bad && lane == 0 && p.status != nullptr) atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
  if (NORM) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // lanes with the same elements: the warp's groups, then the CTA's warps, in that order
      F2x4& dw = t == 0 ? dwq : dwk;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int s = kLanes; s < 32; s <<= 1) {
          dw[e].x += __shfl_xor_sync(0xffffffffu, dw[e].x, s);
          dw[e].y += __shfl_xor_sync(0xffffffffu, dw[e].y, s);
        }
        if ((threadIdx.x & 31) < kLanes) {
          dw_s[threadIdx.x >> 5][8 * lane + 2 * e] = dw[e].x;
          dw_s[threadIdx.x >> 5][8 * lane + 2 * e + 1] = dw[e].y;
        }
      }
      __syncthreads();
      if (threadIdx.x < D) {
        float sum = 0.f;
#pragma unroll
        for (int wp = 0; wp < kNrThreads / 32; ++wp) sum += dw_s[wp][threadIdx.x];
        p.dw_part[(static_cast<long long>(t) * gridDim.x + blockIdx.x) * D + threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
}

constexpr int kRowsAhead = 10;  // 296 CTAs' rows in one turn

// dw = sum over the CTAs' partial rows (q's, then k's): a CTA takes 32 columns of
// one of the two, its 32 warps every 32nd row each, then one warp adds the 32 sums.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int rows, float* dwq, float* dwk) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the partial rows are written
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_k = blockIdx.x >= D / 32;
  const int col = (blockIdx.x - (is_k ? D / 32 : 0)) * 32 + lane;
  const float* from = part + (is_k ? static_cast<long long>(rows) * D : 0);
  float v = 0.f;
  for (int r0 = warp; r0 < rows; r0 += 32 * kRowsAhead) {  // kRowsAhead rows in flight, summed in order
    float t[kRowsAhead];
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k)
      t[k] = r0 + 32 * k < rows ? from[static_cast<long long>(r0 + 32 * k) * D + col] : 0.f;
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) v += t[k];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][lane];
    (is_k ? dwk : dwq)[col] = t;
  }
}

template <int D, bool INTER, bool NORM, bool PAGED>
int launch_fwd_t(NormRopeParams p, int sms, cudaStream_t stream) {
  constexpr unsigned groups = kNrThreads / (D / 8);
  const unsigned tiles = (p.tokens + groups - 1) / groups;
  // As many heads a CTA as leave kFwdCtasPerSm CTAs for every SM: angles and
  // weights are then read once for all of them.
  const unsigned parts = (kFwdCtasPerSm * static_cast<unsigned>(sms) + tiles - 1) / tiles;
  const unsigned all = p.ch.all();
  p.parts = static_cast<int>(parts < all ? parts : all);
  constexpr int smem = Ring<kHeads>::kBytes;
  if (smem > 48 * 1024 && cudaFuncSetAttribute(norm_rope_kernel<D, INTER, NORM, PAGED>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return ATTN_ERR_CUDA;
  norm_rope_kernel<D, INTER, NORM, PAGED><<<tiles * p.parts, kNrThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
template <bool PAGED>
int launch_fwd(const NormRopeParams& p, int d, int interleaved, int sms, cudaStream_t stream) {
  const bool norm = p.w[0] != nullptr;
  if (d == 128)
    return interleaved ? (norm ? launch_fwd_t<128, true, true, PAGED>(p, sms, stream)
                               : launch_fwd_t<128, true, false, PAGED>(p, sms, stream))
                       : (norm ? launch_fwd_t<128, false, true, PAGED>(p, sms, stream)
                               : launch_fwd_t<128, false, false, PAGED>(p, sms, stream));
  return interleaved ? (norm ? launch_fwd_t<64, true, true, PAGED>(p, sms, stream)
                             : launch_fwd_t<64, true, false, PAGED>(p, sms, stream))
                     : (norm ? launch_fwd_t<64, false, true, PAGED>(p, sms, stream)
                             : launch_fwd_t<64, false, false, PAGED>(p, sms, stream));
}

template <int D, bool INTER, bool NORM>
int launch_bwd_t(const NormRopeBwdParams& p, int ctas, float* dwq, float* dwk, cudaStream_t stream) {
  constexpr int smem = Ring<2 * kHeads>::kBytes;
  if (cudaFuncSetAttribute(norm_rope_bwd_kernel<D, INTER, NORM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return ATTN_ERR_CUDA;
  norm_rope_bwd_kernel<D, INTER, NORM><<<ctas, kNrThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (!NORM) return ATTN_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel<D>, static_cast<const float*>(p.dw_part), ctas, dwq, dwk) ==
                 cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

}  // namespace

int norm_rope_chunks(int Hq, int Hkv) { return chunks_of(Hq, Hkv).all(); }

// One wave of CTAs, or one for each step of a small call.
int norm_rope_bwd_ctas(long long tokens, int Hq, int Hkv, int d, int sms) {
  const long long groups = kNrThreads / (d / 8);
  const long long steps = (tokens + groups - 1) / groups * norm_rope_chunks(Hq, Hkv);
  const long long wave = static_cast<long long>(kBwdCtasPerSm) * sms;
  return static_cast<int>(steps < wave ? steps : wave);
}
size_t norm_rope_bwd_workspace(int ctas, int d) { return static_cast<size_t>(ctas) * 2 * d * sizeof(float); }

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
  p.ch = chunks_of(a.Hq, a.Hkv);
  p.w_bf16 = a.w_bf16;
  p.num_slots = num_slots;
  p.eps = a.eps;
  return slots != nullptr ? launch_fwd<true>(p, a.d, a.interleaved, a.sms, stream)
                          : launch_fwd<false>(p, a.d, a.interleaved, a.sms, stream);
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
  const unsigned groups = kNrThreads / (a.d / 8);
  p.tiles = (p.tokens + groups - 1) / groups;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.rd = a.rd;
  p.max_pos = a.max_pos;
  p.ch = chunks_of(a.Hq, a.Hkv);
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
