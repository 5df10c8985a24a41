// Block tables and slot maps of a paged cache, built on the GPU from the
// requests' lengths ("Module 09: Efficient Attention", "The Block Table": a
// sequence of n tokens holds ceil(n / block_size) blocks, token t sits in slot
// t % block_size of block table[t / block_size], and a free list hands the
// blocks out).
//
// extend: sequence b goes from L_b to L_b + n_b tokens and needs
//   c_b = ceil((L_b + n_b) / bs) - ceil(L_b / bs) new blocks.
// The free list is a stack; with off_b = sum_{a < b} c_a the i-th block handed
// out in sequence order is free[F - 1 - i], so entry j of sequence b becomes
// free[F - 1 - (off_b + j - ceil(L_b / bs))]. With cu_b = sum_{a < b} n_a, row
// t of the new tokens belongs to the sequence b with cu_b <= t < cu_{b+1}, sits
// at position L_b + t - cu_b and in slot table[b][pos / bs] * bs + pos % bs.
// release: the blocks of the finished sequences go back on top of the list, in
// sequence order and then in logical order.
//
// Both are prefix sums over the batch, then independent work per new block and
// per row. What bounds them is latency: a step of 64 requests touches 2 KB,
// and the chain lengths -> scan -> free entry -> slot is three dependent memory
// round trips and two scans. So one launch does everything: every CTA scans the
// whole batch for itself (a few KB from L2) and takes a share of the blocks and
// rows, finding a row's sequence by bisection in shared memory. The CTAs form
// one cluster, whose barrier stands between the last read of the lengths and
// the free count and the first write of their new values: they may be updated
// in place. One CTA serves up to kSmallWork rows; eight spread more of them.
// No atomics touch the results, so they are the same on every run.

#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace attn {
namespace {

constexpr int kTableThreads = 1024;
constexpr int kTableCluster = 8;
constexpr int kSmallWork = 4096;
// Consecutive rows or entries of a thread where there are more than threads: one
// bisection and one block's entry serve most (66,000 rows 13.1 -> 10.4 us). With
// fewer each thread takes one: a decode step's rows are of 64 different sequences,
// and four in turn took 6.9 us instead of 4.5.
constexpr unsigned kRun = 4;

struct TableParams {
  const int32_t* seq_lens;
  const int32_t* new_lens;  // extend: new tokens; release: the finished flags
  int32_t* table;
  int32_t* free_blocks;
  const int32_t* num_free;
  int32_t* seq_lens_out;
  int32_t* num_free_out;
  int32_t* cu_q;
  int32_t* positions;
  int32_t* slots;
  int32_t* status;
  int B, num_blocks, block_size, max_blocks, free_cap, max_tokens;
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Inclusive prefix sums over the CTA's threads of a 64-bit and a 32-bit value.
// `warp_sums` holds 32 pairs; *total gets the sums over all threads.
struct Pair {
  long long a;
  int b;
};
__device__ __forceinline__ Pair scan_block(Pair v, Pair* warp_sums, Pair* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, v.a, s);
    const int b = __shfl_up_sync(0xffffffffu, v.b, s);
    if (lane >= s) {
      v.a += a;
      v.b += b;
    }
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  Pair w = warp_sums[lane];  // 32 warps: every warp scans their sums for itself
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, w.a, s);
    const int b = __shfl_up_sync(0xffffffffu, w.b, s);
    if (lane >= s) {
      w.a += a;
      w.b += b;
    }
  }
  const int before = warp > 0 ? warp - 1 : 0;
  const long long ba = __shfl_sync(0xffffffffu, w.a, before);
  const int bb = __shfl_sync(0xffffffffu, w.b, before);
  if (warp > 0) {
    v.a += ba;
    v.b += bb;
  }
  total->a = __shfl_sync(0xffffffffu, w.a, 31);
  total->b = __shfl_sync(0xffffffffu, w.b, 31);
  __syncthreads();  // warp_sums may be written again
  return v;
}

// Blocks that `tokens` tokens fill; unsigned, so that the sum cannot overflow.
__device__ __forceinline__ int blocks_of(int tokens, int bs) {
  return static_cast<int>((static_cast<unsigned>(tokens) + static_cast<unsigned>(bs) - 1u) / static_cast<unsigned>(bs));
}
// The mark of a sequence that could not be extended, and the length behind it.
__device__ __forceinline__ int failed_mark(int len) { return -1 - len; }

// The last index b in [0, n) with start[b] <= x (start[0] = 0, ascending):
// of equal starts the last, so sequences with nothing are never found.
__device__ __forceinline__ int last_at_or_below(const int* start, int n, int x) {
  int lo = 0, hi = n;  // start[lo] <= x, and start[hi] > x or hi = n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Shared memory: per sequence the row start, the block start and the length
// (negative: the sequence failed and gets nothing; what its length becomes).
template <bool RELEASE>
__global__ void __launch_bounds__(kTableThreads, 1) paged_table_kernel(const TableParams p) {
  extern __shared__ int32_t table_smem[];
  __shared__ Pair warp_sums[32];
  __shared__ int taken;  // blocks handed out: up to the last sequence that got its own
  int* cu = table_smem;
  int* off = cu + p.B;
  int* len = off + p.B;
  const int tid = threadIdx.x;
  const int rank = blockIdx.x, ranks = gridDim.x;  // the grid is one cluster
  const int bs = p.block_size;
  const long long table_tokens = static_cast<long long>(p.max_blocks) * bs;

  if (tid == 0) taken = 0;
  // plain loads, not the read-only path: these may be updated in place below
  const int F0 = *p.num_free;
  bool flag = F0 < 0 || F0 > p.free_cap;
  const int F = flag ? (RELEASE ? p.free_cap : 0) : F0;  // a bad count: nothing to take, no room to give back
  Pair run{0, 0};
  __syncthreads();
  for (int base = 0; base < p.B; base += kTableThreads) {
    const int b = base + tid;
    int L = 0, n = 0, c = 0;
    bool ok = true;
    if (b < p.B) {
      L = p.seq_lens[b];
      n = p.new_lens[b];
      if (RELEASE) {
        n = n != 0;
        if (n) {  // a running sequence is passed through as it is
          const int held = L < 0 ? failed_mark(L) : L;
          ok = held <= table_tokens;
          if (ok) c = blocks_of(held, bs);
        }
      } else {
        ok = n >= 0 && L >= 0 && static_cast<long long>(L) + n <= table_tokens;
        if (n < 0) n = 0;
        if (ok) c = blocks_of(L + n, bs) - blocks_of(L, bs);
      }
    }
    Pair total;
    Pair v = scan_block(Pair{RELEASE ? 0 : n, c}, warp_sums, &total);
    v.a += run.a;
    v.b += run.b;
    run.a += total.a;
    run.b += total.b;
    if (b < p.B) {
      if (!RELEASE) {
        // out of blocks or rows: inclusive sums, so everything after the first that does not fit fails too
        if (ok && c > 0 && v.b > F) ok = false;
        if (n > 0 && v.a > p.max_tokens) ok = false;
        if (ok && c > 0) atomicMax(&taken, v.b);
        const long long start = v.a - n;
        cu[b] = static_cast<int>(start < p.max_tokens ? start : p.max_tokens);
      }
      off[b] = v.b - c;
      len[b] = RELEASE ? (n ? 0 : L) : (ok || L < 0 ? L : failed_mark(L));
      flag |= !ok;
    }
  }
  const int rows = static_cast<int>(run.a < p.max_tokens ? run.a : p.max_tokens);
  __syncthreads();
  // every CTA has read the lengths and the free count: they may be written now
  cluster_barrier();

  // unsigned: the last step past the end may not wrap into negative indexes
  const unsigned t0 = rank * kTableThreads + tid, step = ranks * kTableThreads, B = p.B;
  if (RELEASE) {
    for (unsigned b = t0; b < B; b += step) p.seq_lens_out[b] = len[b];
    const long long room = p.free_cap - F;
    const int given = static_cast<int>(run.b < room ? run.b : room);
    flag |= run.b > room;
    if (t0 == 0) *p.num_free_out = F0 + given;
    const unsigned n = given, run = n <= step ? 1 : kRun;
    for (unsigned i0 = run * t0; i0 < n; i0 += run * step) {
      int b = last_at_or_below(off, p.B, static_cast<int>(i0)), e[kRun];
#pragma unroll
      for (unsigned k = 0; k < kRun; ++k) {
        const unsigned i = i0 + k;
        e[k] = 0;
        if (k < run && i < n) {
          // of equal starts the last: sequences that give nothing are passed over
          while (b + 1 < p.B && static_cast<unsigned>(off[b + 1]) <= i) ++b;
          e[k] = p.table[static_cast<size_t>(b) * p.max_blocks + (i - off[b])];
        }
      }
#pragma unroll
      for (unsigned k = 0; k < kRun; ++k) {
        if (k < run && i0 + k < n) {
          flag |= e[k] < 0 || e[k] >= p.num_blocks;
          p.free_blocks[F + i0 + k] = e[k];
        }
      }
    }
  } else {
    if (t0 == 0) *p.num_free_out = F0 - taken;
    for (unsigned b = t0; b < B; b += step) {
      p.cu_q[b] = cu[b];
      const int end = b + 1 < B ? cu[b + 1] : rows;
      // a sequence that failed stays marked: nothing may read its cache as if it had grown
      p.seq_lens_out[b] = len[b] < 0 ? len[b] : len[b] + (end - cu[b]);
    }
    if (t0 == 0) p.cu_q[p.B] = rows;
    for (unsigned i = t0; i < static_cast<unsigned>(taken); i += step) {
      const int b = last_at_or_below(off, p.B, static_cast<int>(i));
      const int e = p.free_blocks[F - 1 - i];
      const bool good = e >= 0 && e < p.num_blocks;
      flag |= !good;
      p.table[static_cast<size_t>(b) * p.max_blocks + blocks_of(len[b], bs) + (i - off[b])] = good ? e : -1;
    }
    const unsigned n = p.max_tokens, filled = rows, run = n <= step ? 1 : kRun;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15u) == 0;
    for (unsigned r0 = run * t0; r0 < n; r0 += run * step) {
      int pos[kRun], slot[kRun];
      int b = -1, m = 0, blk = 0, at = 0, have = 0, e = -1;  // the row's sequence, position, block and its entry
      unsigned end = 0;                                      // the sequence's last row
#pragma unroll
      for (unsigned k = 0; k < kRun; ++k) {
        const unsigned t = r0 + k;
        pos[k] = 0;
        slot[k] = -1;
        if (k >= run || t >= filled) continue;
        bool look = true;
        if (t >= end) {
          if (b < 0) b = last_at_or_below(cu, p.B, static_cast<int>(t));
          while (b + 1 < p.B && static_cast<unsigned>(cu[b + 1]) <= t) ++b;
          end = b + 1 < p.B ? cu[b + 1] : rows;
          m = len[b] + (static_cast<int>(t) - cu[b]);
          have = len[b] < 0 ? 0 : blocks_of(len[b], bs);
          blk = m / bs;
          at = m - blk * bs;
        } else {
          ++m;
          look = ++at == bs;
          if (look) {
            at = 0;
            ++blk;
          }
        }
        if (len[b] < 0) continue;
        // the block the sequence stopped in, or one handed out above
        if (look)
          e = blk < have ? p.table[static_cast<size_t>(b) * p.max_blocks + blk]
                         : p.free_blocks[F - 1 - (off[b] + blk - have)];
        const bool good = e >= 0 && e < p.num_blocks;
        flag |= !good;
        pos[k] = m;
        slot[k] = good ? e * bs + at : -1;
      }
      if (wide && run == kRun && r0 + kRun <= n) {
        *reinterpret_cast<int4*>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (unsigned k = 0; k < kRun; ++k) {
          if (k < run && r0 + k < n) {
            p.positions[r0 + k] = pos[k];
            p.slots[r0 + k] = slot[k];
          }
        }
      }
    }
  }
  if (flag && p.status != nullptr) atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
}

template <bool RELEASE>
int launch_table(const TableParams& p, long long work, cudaStream_t stream) {
  const int smem = 3 * p.B * static_cast<int>(sizeof(int32_t));
  if (smem > 48 * 1024 - 1024 &&  // more than a kernel may have unasked
      cudaFuncSetAttribute(paged_table_kernel<RELEASE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           3 * kMaxTableSeqs * static_cast<int>(sizeof(int32_t))) != cudaSuccess)
    return ATTN_ERR_CUDA;
  const unsigned ctas = work > kSmallWork ? kTableCluster : 1;
  if (ctas == 1) {  // a cluster of its own, and a cheaper launch
    paged_table_kernel<RELEASE><<<1, kTableThreads, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTableThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_table_kernel<RELEASE>, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

int launch_paged_extend(const int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table,
                        const int32_t* free_blocks, const int32_t* num_free, int32_t* seq_lens_out,
                        int32_t* num_free_out, int32_t* cu_q, int32_t* positions, int32_t* slots, int B,
                        int num_blocks, int block_size, int max_blocks_per_seq, int free_capacity, int max_tokens,
                        int32_t* status, cudaStream_t stream) {
  const TableParams p{seq_lens, new_lens, block_table, const_cast<int32_t*>(free_blocks), num_free, seq_lens_out,
                      num_free_out, cu_q, positions, slots, status, B, num_blocks, block_size, max_blocks_per_seq,
                      free_capacity, max_tokens};
  return launch_table<false>(p, static_cast<long long>(max_tokens), stream);
}

int launch_paged_release(const int32_t* seq_lens, const int32_t* finished, const int32_t* block_table,
                         int32_t* free_blocks, const int32_t* num_free, int32_t* seq_lens_out, int32_t* num_free_out,
                         int B, int num_blocks, int block_size, int max_blocks_per_seq, int free_capacity,
                         int32_t* status, cudaStream_t stream) {
  const TableParams p{seq_lens, finished, const_cast<int32_t*>(block_table), free_blocks, num_free, seq_lens_out,
                      num_free_out, nullptr, nullptr, nullptr, status, B, num_blocks, block_size, max_blocks_per_seq,
                      free_capacity, 0};
  // how many blocks go back is known on the device only: at most all of the table's
  return launch_table<true>(p, static_cast<long long>(B) * max_blocks_per_seq, stream);
}

}  // namespace attn
