// The block pool on the GPU: growing every sequence of a batch by its new
// tokens (block tables, slots and positions from lengths alone), and giving
// the blocks of finished sequences back.
//
// The pool is a stack of free block ids, free_list[0 .. count). With
// had_b = ceil(L_b / bs) and has_b = ceil((L_b + n_b) / bs), sequence b needs
// has_b - had_b blocks; with e the exclusive prefix sum of these over b,
//   table[b][had_b + i] = free_list[count - 1 - (e_b + i)],
// and with s the exclusive prefix sum of n, row t of [s_b, s_{b+1}) is the
// token at position p = L_b + t - s_b, in slot table[b][p / bs] * bs + p % bs.
// Releasing pushes table[b][keep_b .. had_b) at count + e_b in the same way.
//
// Both are integer work with no arithmetic to speak of: a small step is bound
// by the launch and three dependent round trips (lengths, a table or free
// entry, the stores), a large one by the stores of its slots. So one launch
// does everything: every CTA scans the whole batch (two words a sequence from
// L2, at most 4096 sequences) into shared memory and then writes its share of
// the rows and table entries, found by binary search in the prefix sums. No
// CTA waits for another. Where the lengths or the pool's state are updated in
// place, the CTA that is last to have read them (a ticket in the pool's own
// state) writes them.
#include "pa_internal.h"
#include "ptx.cuh"
#include "step_ops.h"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

// Inclusive sums of (x, y) over the block; *tx, *ty receive the totals.
__device__ __forceinline__ void block_scan2(long long& x, int& y, long long* tx, int* ty) {
  __shared__ long long s_x[kWarps];
  __shared__ int s_y[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(kFull, x, o);
    const int v = __shfl_up_sync(kFull, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    s_x[warp] = x;
    s_y[warp] = y;
  }
  __syncthreads();
  long long bx = 0, ax = 0;
  int by = 0, ay = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) {
      bx = ax;
      by = ay;
    }
    ax += s_x[w];
    ay += s_y[w];
  }
  x += bx;
  y += by;
  *tx = ax;
  *ty = ay;
  __syncthreads();  // the sums are reused by the next round
}

// The error bits of any thread of the block.
__device__ __forceinline__ int block_or(int bits) {
  int r = 0;
  for (const int bit : {PA_DEVERR_SEQ_LEN, PA_DEVERR_POOL, PA_DEVERR_TOKENS})
    r |= __syncthreads_or(bits & bit) ? bit : 0;
  return r;
}

// The index b in [0, B) with s[b] <= x < s[b + 1], for s[0] <= x < s[B]
// (sequences with nothing are skipped).
__device__ __forceinline__ int row_of(const int* s, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// True for the one CTA that may overwrite what every CTA has read: the first
// one where nothing is updated in place, else the last to arrive here.
__device__ __forceinline__ bool commit_turn(bool in_place, int32_t* ticket) {
  if (!in_place || gridDim.x == 1) return blockIdx.x == 0;
  __shared__ int s_last;
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  return s_last != 0;
}

struct Share {
  int lo, hi;
};
// This CTA's share of n items, in multiples of `unit`.
__device__ __forceinline__ Share share_of(int n, int unit) {
  const long long units = (static_cast<long long>(n) + unit - 1) / unit;
  const long long per = (units + gridDim.x - 1) / gridDim.x * unit;
  const long long lo = per * blockIdx.x;
  Share s;
  s.lo = static_cast<int>(min(lo, static_cast<long long>(n)));
  s.hi = static_cast<int>(min(lo + per, static_cast<long long>(n)));
  return s;
}

__global__ void __launch_bounds__(kThreads) pool_extend_kernel(const PoolExtendArgs a) {
  extern __shared__ int s_dyn[];
  int* s_tok = s_dyn;             // [B + 1] exclusive prefix of the new tokens
  int* s_blk = s_tok + a.B + 1;   // [B + 1] exclusive prefix of the new blocks
  int* s_len = s_blk + a.B + 1;   // [B] lengths before the step
  const int tid = threadIdx.x;
  griddep_wait();  // everything read here may come from the previous kernel
  const long long cap = static_cast<long long>(a.MB) * a.bs;
  const int count = a.state[0];
  int bad = 0;
  long long tok = 0;
  int blk = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int L = 0, n = 0;
    if (b < a.B) {
      L = a.lens[b];
      n = a.fresh[b];
      if (n < 0) bad |= PA_DEVERR_TOKENS;
      if (L < 0 || static_cast<long long>(L) + n > cap) bad |= PA_DEVERR_SEQ_LEN;
      s_len[b] = L;
      if (bad) n = 0, L = 0;  // the step is refused below; keep the sums in range
    }
    long long x = n, tx;
    int y = (L + n + a.bs - 1) / a.bs - (L + a.bs - 1) / a.bs, ty;
    const int y0 = y;
    block_scan2(x, y, &tx, &ty);
    if (b < a.B) {
      s_tok[b] = static_cast<int>(min(tok + x - n, static_cast<long long>(a.T)));
      s_blk[b] = blk + y - y0;
    }
    tok += tx;
    blk += ty;
  }
  if (tok > a.T) bad |= PA_DEVERR_TOKENS;
  if (count < 0 || count > a.NF || blk > count) bad |= PA_DEVERR_POOL;
  bad = block_or(bad);
  const bool ok = bad == 0;
  const int ntok = ok ? static_cast<int>(tok) : 0, nblk = ok ? blk : 0;
  if (tid == 0) {
    s_tok[a.B] = ntok;
    s_blk[a.B] = nblk;
  }
  __syncthreads();

  // new table entries
  const Share sb = share_of(nblk, 32);
  for (int i = sb.lo + tid; i < sb.hi; i += kThreads) {
    const int b = row_of(s_blk, a.B, i);
    const int had = (s_len[b] + a.bs - 1) / a.bs;
    const int id = a.free_list[count - 1 - i];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.NF)) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
    a.tables[static_cast<size_t>(b) * a.MB + had + (i - s_blk[b])] = id;
  }

  // slots and positions, four rows a thread: one search, then along the rows
  const Share st = share_of(a.T, 4 * 32);
  for (int t0 = st.lo + 4 * tid; t0 < st.hi; t0 += 4 * kThreads) {
    long long slot[4];
    int pos[4];
    int b = -1, end = 0, base = 0, had = 0, cur = -1;
    long long first = -1;  // first slot of block `cur` of sequence b
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j;
      slot[j] = -1;
      pos[j] = 0;
      if (t >= ntok) continue;
      if (b < 0 || t >= end) {
        b = row_of(s_tok, a.B, t);
        end = s_tok[b + 1];
        base = s_len[b] - s_tok[b];
        had = (s_len[b] + a.bs - 1) / a.bs;
        cur = -1;
      }
      const int p = base + t;
      const int k = p / a.bs;
      if (k != cur) {
        cur = k;
        const int id = k < had ? a.tables[static_cast<size_t>(b) * a.MB + k]
                               : a.free_list[count - 1 - (s_blk[b] + k - had)];
        const bool fine = static_cast<unsigned>(id) < static_cast<unsigned>(a.NF);
        if (!fine) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
        first = fine ? static_cast<long long>(id) * a.bs : -1;
      }
      slot[j] = first < 0 ? -1 : first + (p - k * a.bs);
      pos[j] = p;
    }
    if (a.wide && t0 + 4 <= a.T) {
      longlong2* ds = reinterpret_cast<longlong2*>(a.slots + t0);
      ds[0] = make_longlong2(slot[0], slot[1]);
      ds[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t0 + j < a.T) {
          a.slots[t0 + j] = slot[j];
          a.positions[t0 + j] = pos[j];
        }
    }
  }

  if (!commit_turn(a.in_place, a.state + 1)) return;
  for (int b = tid; b <= a.B; b += kThreads) {
    const int s = ok ? s_tok[b] : 0;
    a.query_start[b] = s;
    if (b < a.B) a.lens_out[b] = s_len[b] + (ok ? s_tok[b + 1] - s : 0);
  }
  if (tid == 0) {
    if (bad) atomicOr(a.err, bad);
    a.state_out[0] = count - nblk;
    a.state_out[1] = 0;
  }
}

__global__ void __launch_bounds__(kThreads) pool_release_kernel(const PoolReleaseArgs a) {
  extern __shared__ int s_dyn[];
  int* s_blk = s_dyn;             // [B + 1] exclusive prefix of the released blocks
  int* s_keep = s_blk + a.B + 1;  // [B] first block of each sequence that is given back
  int* s_len = s_keep + a.B;      // [B] lengths before the call
  const int tid = threadIdx.x;
  griddep_wait();
  const long long cap = static_cast<long long>(a.MB) * a.bs;
  const int count = a.state[0];
  int bad = 0, blk = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int y = 0;
    if (b < a.B) {
      const int L = a.lens[b];
      const bool gone = a.released[b] != 0;
      int keep = 0;
      if (gone) {
        if (L < 0 || L > cap) {
          bad |= PA_DEVERR_SEQ_LEN;
        } else {
          const int sh = a.shared ? a.shared[b] : 0;
          keep = sh > 0 ? sh / a.bs : 0;
          y = max((L + a.bs - 1) / a.bs - keep, 0);
        }
      }
      s_keep[b] = keep;
      s_len[b] = L;
    }
    const int y0 = y;
    long long x = 0, tx;
    int ty;
    block_scan2(x, y, &tx, &ty);
    if (b < a.B) s_blk[b] = blk + y - y0;
    blk += ty;
  }
  if (count < 0 || static_cast<long long>(count) + blk > a.NF) bad |= PA_DEVERR_POOL;
  bad = block_or(bad);
  const bool ok = bad == 0;
  const int nblk = ok ? blk : 0;
  if (tid == 0) s_blk[a.B] = nblk;
  __syncthreads();

  // a warp copies runs of 32 entries; its lanes search again only where a
  // sequence ends
  const Share sb = share_of(nblk, 32);
  int b = -1;
  for (int i = sb.lo + tid; i < sb.hi; i += kThreads) {
    if (b < 0 || i >= s_blk[b + 1]) b = row_of(s_blk, a.B, i);
    const int id = a.tables[static_cast<size_t>(b) * a.MB + s_keep[b] + (i - s_blk[b])];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.NF)) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
    a.free_list[count + i] = id;
  }

  if (!commit_turn(a.in_place, a.state + 1)) return;
  for (int r = tid; r < a.B; r += kThreads)
    a.lens_out[r] = ok && a.released[r] != 0 ? 0 : s_len[r];
  if (tid == 0) {
    if (bad) atomicOr(a.err, bad);
    a.state_out[0] = count + nblk;
    a.state_out[1] = 0;
  }
}

// CTAs for `items` outputs of `per` each: one where they fit one CTA (no
// ticket, no repeated scan), at most two an SM.
int grid_for(long long items, long long per, int num_sms) {
  const long long g = (items + per - 1) / per;
  return static_cast<int>(g < 1 ? 1 : (g > 2ll * num_sms ? 2ll * num_sms : g));
}

template <typename Args>
cudaError_t launch(void (*fn)(const Args), const Args& a, int grid, size_t smem, cudaStream_t s) {
  if (smem > 48 * 1024) {  // large batches: the per-sequence prefixes
    const cudaError_t e =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace

cudaError_t pool_extend_launch(const PoolExtendArgs& a, int num_sms, cudaStream_t s) {
  const size_t smem = (3 * static_cast<size_t>(a.B) + 2) * sizeof(int);
  return launch(pool_extend_kernel, a, grid_for(a.T, 4 * kThreads, num_sms), smem, s);
}

cudaError_t pool_release_launch(const PoolReleaseArgs& a, int num_sms, cudaStream_t s) {
  const size_t smem = (3 * static_cast<size_t>(a.B) + 1) * sizeof(int);
  // the host knows only what the tables could hold
  const long long most = static_cast<long long>(a.B) * a.MB;
  return launch(pool_release_kernel, a, grid_for(most, 4 * kThreads, num_sms), smem, s);
}

}  // namespace pa
