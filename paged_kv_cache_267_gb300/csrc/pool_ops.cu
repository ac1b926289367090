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
// entry, the stores), a large one by the scan and the stores of its slots (64
// sequences of a token each 3.1 us in a graph, 2^20 rows of 256 prompts 6.8 us,
// 917,000 entries of 4096 sequences given back 6.8 us). So one launch
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
constexpr int kMaxRows = 4096 / kThreads;  // of the batch, a thread
constexpr int kMostShared = (3 * kThreads * kMaxRows + 2) * 4;  // bytes, at the largest batch
constexpr unsigned kFull = 0xffffffffu;
// Token sums saturate here: more than any call accepts, and the sum of two
// such values still fits 32 bits.
constexpr unsigned kManyTokens = (1u << 30) + 1;

__device__ __forceinline__ unsigned add_tokens(unsigned x, unsigned y) {
  return min(x + y, kManyTokens);
}

struct Sums {
  unsigned tok;  // saturating
  int blk;
  int bad;       // error bits of any thread
};

// Exclusive sums of the threads' tokens and blocks over the block; *all
// receives the totals. One barrier: every warp scans the warps' totals.
__device__ __forceinline__ Sums block_sums(Sums v, Sums* all) {
  __shared__ unsigned s_t[kWarps];
  __shared__ int s_b[kWarps], s_e[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned t = v.tok;
  int b = v.blk;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(kFull, t, o);
    const int z = __shfl_up_sync(kFull, b, o);
    if (lane >= o) {
      t = add_tokens(t, y);
      b += z;
    }
  }
  const int bad = __reduce_or_sync(kFull, v.bad);
  if (lane == 31) {
    s_t[warp] = t;
    s_b[warp] = b;
    s_e[warp] = bad;
  }
  // the lane before: this thread's sums without itself
  unsigned t0 = __shfl_up_sync(kFull, t, 1);
  int b0 = __shfl_up_sync(kFull, b, 1);
  if (lane == 0) t0 = 0, b0 = 0;
  __syncthreads();
  unsigned wt = lane < kWarps ? s_t[lane] : 0u;
  int wb = lane < kWarps ? s_b[lane] : 0;
  all->bad = __reduce_or_sync(kFull, lane < kWarps ? s_e[lane] : 0);
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const unsigned y = __shfl_up_sync(kFull, wt, o);
    const int z = __shfl_up_sync(kFull, wb, o);
    if (lane >= o) {
      wt = add_tokens(wt, y);
      wb += z;
    }
  }
  all->tok = __shfl_sync(kFull, wt, kWarps - 1);
  all->blk = __shfl_sync(kFull, wb, kWarps - 1);
  const unsigned pt = __shfl_sync(kFull, wt, warp > 0 ? warp - 1 : 0);
  const int pb = __shfl_sync(kFull, wb, warp > 0 ? warp - 1 : 0);
  if (warp > 0) {
    t0 = add_tokens(t0, pt);
    b0 += pb;
  }
  return Sums{t0, b0, 0};
}

// Turns the counts s_tok[0 .. B) (null: none) and s_blk[0 .. B) into their
// exclusive prefix sums; the block's error bits and totals come back. Rows are
// loaded by the callers in coalesced order; here a thread takes consecutive
// ones, so that one scan serves any batch.
__device__ __forceinline__ Sums scan_rows(int* s_tok, int* s_blk, int B, int bad) {
  const int per = (B + kThreads - 1) / kThreads;
  const int lo = min(static_cast<int>(threadIdx.x) * per, B), hi = min(lo + per, B);
  Sums mine = {0u, 0, bad};
  for (int b = lo; b < hi; ++b) {
    if (s_tok) mine.tok = add_tokens(mine.tok, static_cast<unsigned>(s_tok[b]));
    mine.blk += s_blk[b];
  }
  Sums all;
  const Sums before = block_sums(mine, &all);
  unsigned t = before.tok;
  int k = before.blk;
  for (int b = lo; b < hi; ++b) {
    if (s_tok) {
      const unsigned n = static_cast<unsigned>(s_tok[b]);
      s_tok[b] = static_cast<int>(t);
      t = add_tokens(t, n);
    }
    const int n = s_blk[b];
    s_blk[b] = k;
    k += n;
  }
  return all;
}

// The index b in [lo, B) with s[b] <= x < s[b + 1], for s[lo] <= x < s[B]
// (sequences with nothing are skipped).
__device__ __forceinline__ int row_of(const int* s, int B, int x, int lo = 0) {
  int hi = B;
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
    // (wraps to zero for the next call, whichever of the two is in place)
    s_last = atomicInc(reinterpret_cast<unsigned*>(ticket), gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  return s_last != 0;
}

// n / d for n < 2^31 by the multiplication the host prepared: with l =
// ceil(log2 d) and m = ceil(2^(31 + l) / d), m d - 2^(31 + l) < 2^l, so the
// quotient n m / 2^(31 + l) exceeds n / d by less than 1 / d.
__device__ __forceinline__ int quot(int n, const FastDiv& f) {
  return static_cast<int>(__umulhi(static_cast<unsigned>(n), f.mul) >> f.shift);
}

struct Share {
  int lo, hi;
};
// This CTA's share of n <= 2^31 - 2^16 items, in multiples of `unit`.
__device__ __forceinline__ Share share_of(int n, int unit) {
  const unsigned units = (static_cast<unsigned>(n) + unit - 1) / unit;
  const unsigned per = (units + gridDim.x - 1) / gridDim.x * unit;
  const unsigned long long lo = static_cast<unsigned long long>(per) * blockIdx.x;
  Share s;
  s.lo = static_cast<int>(min(lo, static_cast<unsigned long long>(n)));
  s.hi = static_cast<int>(min(lo + per, static_cast<unsigned long long>(n)));
  return s;
}

// The step's scanned state, for the writers of its rows.
struct Step {
  const int *tok, *blk, *len;
  int count, ntok;
};

// Slots and positions of rows [t0, t0 + N): one search, then along the rows.
// The rows belong to sequences [b_lo, b_hi).
template <int N>
__device__ __forceinline__ void write_rows(const PoolExtendArgs& a, const Step& s, int t0, int b_lo,
                                           int b_hi) {
  long long slot[N];
  int pos[N];
  int b = -1, end = 0, base = 0, had = 0, cur = -1;
  long long first = -1;  // first slot of block `cur` of sequence b
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int t = t0 + j;
    slot[j] = -1;
    pos[j] = 0;
    if (t >= s.ntok) continue;
    if (b < 0 || t >= end) {
      b = row_of(s.tok, b_hi, t, b_lo);
      end = s.tok[b + 1];
      base = s.len[b] - s.tok[b];
      had = quot(s.len[b] + a.bs - 1, a.div);
      cur = -1;
    }
    const int p = base + t;
    const int k = quot(p, a.div);
    if (k != cur) {
      cur = k;
      const int id = k < had ? a.tables[static_cast<size_t>(b) * a.MB + k]
                             : a.free_list[s.count - 1 - (s.blk[b] + k - had)];
      const bool fine = static_cast<unsigned>(id) < static_cast<unsigned>(a.NF);
      if (!fine) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
      first = fine ? static_cast<long long>(id) * a.bs : -1;
    }
    slot[j] = first < 0 ? -1 : first + (p - k * a.bs);
    pos[j] = p;
  }
  if constexpr (N == 4) {
    if (a.wide && t0 + 4 <= a.T) {
      longlong2* ds = reinterpret_cast<longlong2*>(a.slots + t0);
      ds[0] = make_longlong2(slot[0], slot[1]);
      ds[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (t0 + j < a.T) {
      a.slots[t0 + j] = slot[j];
      a.positions[t0 + j] = pos[j];
    }
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
  int row_len[kMaxRows], row_new[kMaxRows];  // rows tid, tid + kThreads, ...
#pragma unroll
  for (int j = 0; j < kMaxRows; ++j) {
    const int b = j * kThreads + tid;
    row_len[j] = b < a.B ? a.lens[b] : 0;
    row_new[j] = b < a.B ? a.fresh[b] : 0;
  }
  int bad = 0;
#pragma unroll
  for (int j = 0; j < kMaxRows; ++j) {
    const int b = j * kThreads + tid;
    if (b >= a.B) break;
    const int L = row_len[j], n = row_new[j];
    int row_bad = n < 0 ? PA_DEVERR_TOKENS : 0;
    if (L < 0 || static_cast<long long>(L) + n > cap) row_bad |= PA_DEVERR_SEQ_LEN;
    bad |= row_bad;
    // a bad row refuses the step below; it counts nothing here
    s_len[b] = L;
    s_tok[b] = row_bad ? 0 : n;
    s_blk[b] = row_bad ? 0 : quot(L + n + a.bs - 1, a.div) - quot(L + a.bs - 1, a.div);
  }
  __syncthreads();
  const Sums all = scan_rows(s_tok, s_blk, a.B, bad);
  bad = all.bad;
  if (all.tok > static_cast<unsigned>(a.T)) bad |= PA_DEVERR_TOKENS;
  if (count < 0 || count > a.NF || all.blk > count) bad |= PA_DEVERR_POOL;
  const bool ok = bad == 0;
  const int ntok = ok ? static_cast<int>(all.tok) : 0, nblk = ok ? all.blk : 0;
  if (tid == 0) {
    s_tok[a.B] = ntok;
    s_blk[a.B] = nblk;
  }
  __syncthreads();

  // new table entries
  const Share sb = share_of(nblk, 32);
  for (int i = sb.lo + tid; i < sb.hi; i += kThreads) {
    const int b = row_of(s_blk, a.B, i);
    const int had = quot(s_len[b] + a.bs - 1, a.div);
    const int id = a.free_list[count - 1 - i];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.NF)) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
    a.tables[static_cast<size_t>(b) * a.MB + had + (i - s_blk[b])] = id;
  }

  // Rows: one a thread where that is one round (decode steps, whose rows are
  // all of different sequences: four in a row would wait for four table
  // entries in turn, 5.8 us against 3.6 us a step of 64), else four.
  const Step step = {s_tok, s_blk, s_len, count, ntok};
  if (a.T <= static_cast<int>(gridDim.x) * kThreads) {
    const int t = blockIdx.x * kThreads + tid;
    if (t < a.T) write_rows<1>(a, step, t, 0, a.B);
  } else {
    const Share st = share_of(a.T, 4 * 32);
    const int last = min(st.hi, ntok) - 1;  // the share meets few sequences
    const int b_lo = st.lo <= last ? row_of(s_tok, a.B, st.lo) : 0;
    const int b_hi = st.lo <= last ? row_of(s_tok, a.B, last, b_lo) + 1 : 0;
    for (int t0 = st.lo + 4 * tid; t0 < st.hi; t0 += 4 * kThreads)
      write_rows<4>(a, step, t0, b_lo, b_hi);
  }

  if (!commit_turn(a.in_place, a.state + 1)) return;
#pragma unroll
  for (int j = 0; j < kMaxRows; ++j) {
    const int b = j * kThreads + tid;
    if (b >= a.B) break;
    a.query_start[b] = ok ? s_tok[b] : 0;
    a.lens_out[b] = row_len[j] + (ok ? row_new[j] : 0);
  }
  if (tid == 0) {
    a.query_start[a.B] = ntok;
    if (bad) atomicOr(a.err, bad);
    a.state_out[0] = count - nblk;
    a.state_out[1] = 0;
  }
}

__global__ void __launch_bounds__(kThreads) pool_release_kernel(const PoolReleaseArgs a) {
  extern __shared__ int s_dyn[];
  int* s_blk = s_dyn;             // [B + 1] exclusive prefix of the released blocks
  int* s_keep = s_blk + a.B + 1;  // [B] first block of each sequence that is given back
  const int tid = threadIdx.x;
  griddep_wait();
  const long long cap = static_cast<long long>(a.MB) * a.bs;
  const int count = a.state[0];
  int row_len[kMaxRows], row_gone[kMaxRows], row_kept[kMaxRows];  // rows tid, tid + kThreads, ...
#pragma unroll
  for (int j = 0; j < kMaxRows; ++j) {
    const int b = j * kThreads + tid;
    row_len[j] = b < a.B ? a.lens[b] : 0;
    row_gone[j] = b < a.B ? a.released[b] : 0;
    row_kept[j] = b < a.B && a.shared ? a.shared[b] : 0;
  }
  int bad = 0;
#pragma unroll
  for (int j = 0; j < kMaxRows; ++j) {
    const int b = j * kThreads + tid;
    if (b >= a.B) break;
    const int L = row_len[j];
    int keep = 0, n = 0;
    if (row_gone[j] != 0) {
      if (L < 0 || L > cap) {
        bad |= PA_DEVERR_SEQ_LEN;
      } else {
        keep = row_kept[j] > 0 ? quot(row_kept[j], a.div) : 0;
        n = max(quot(L + a.bs - 1, a.div) - keep, 0);
      }
    }
    s_keep[b] = keep;
    s_blk[b] = n;
  }
  __syncthreads();
  const Sums all = scan_rows(nullptr, s_blk, a.B, bad);
  bad = all.bad;
  if (count < 0 || static_cast<long long>(count) + all.blk > a.NF) bad |= PA_DEVERR_POOL;
  const bool ok = bad == 0;
  const int nblk = ok ? all.blk : 0;
  if (tid == 0) s_blk[a.B] = all.blk;
  __syncthreads();

  // This CTA's share of the entries, a sequence's part a warp, 8 x 32 entries
  // with their loads in flight together. (Searching the sequence of every
  // entry instead cost most of the call, 16 us for 917,000 entries of 4096
  // sequences.)
  constexpr int kRun = 8;
  const Share sb = share_of(nblk, 32);
  if (sb.lo < sb.hi) {
    const int lane = tid & 31;
    for (int b = row_of(s_blk, a.B, sb.lo) + (tid >> 5); b < a.B; b += kWarps) {
      const int e0 = s_blk[b], i1 = min(s_blk[b + 1], sb.hi);
      if (e0 >= sb.hi) break;
      const int32_t* entry = a.tables + static_cast<size_t>(b) * a.MB + s_keep[b] - e0;
      for (int i0 = max(e0, sb.lo) + lane; i0 < i1; i0 += 32 * kRun) {
        int id[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) id[j] = i0 + 32 * j < i1 ? entry[i0 + 32 * j] : 0;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
          if (i0 + 32 * j >= i1) break;
          if (static_cast<unsigned>(id[j]) >= static_cast<unsigned>(a.NF))
            atomicOr(a.err, PA_DEVERR_BLOCK_ID);
          a.free_list[count + i0 + 32 * j] = id[j];
        }
      }
    }
  }

  if (!commit_turn(a.in_place, a.state + 1)) return;
#pragma unroll
  for (int j = 0; j < kMaxRows; ++j) {
    const int b = j * kThreads + tid;
    if (b >= a.B) break;
    a.lens_out[b] = ok && row_gone[j] != 0 ? 0 : row_len[j];
  }
  if (tid == 0) {
    if (bad) atomicOr(a.err, bad);
    a.state_out[0] = count + nblk;
    a.state_out[1] = 0;
  }
}

// CTAs for `items` outputs of `per` each: one where they fit one CTA (no
// ticket, no repeated scan), at most `most`, which is as many as the SMs hold at
// once or fewer (every CTA scans the batch).
int grid_for(long long items, long long per, int most) {
  const long long g = (items + per - 1) / per;
  return static_cast<int>(g < 1 ? 1 : (g > most ? most : g));
}

template <typename Args>
cudaError_t launch(void (*fn)(const Args), const Args& a, int grid, size_t smem, cudaStream_t s) {
  // Large batches: the per-sequence prefixes. Without asking, a CTA has 48 KB, its
  // static arrays (0.2 KB) among them. (One value, whichever thread sets it.)
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
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
  return launch(pool_extend_kernel, a, grid_for(a.T, 4 * kThreads, 2 * num_sms), smem, s);
}

cudaError_t pool_release_launch(const PoolReleaseArgs& a, int num_sms, cudaStream_t s) {
  const size_t smem = (2 * static_cast<size_t>(a.B) + 1) * sizeof(int);
  // the host knows only what the tables could hold
  const long long most = static_cast<long long>(a.B) * a.MB;
  return launch(pool_release_kernel, a, grid_for(most, 4 * kThreads, num_sms), smem, s);
}

}  // namespace pa
