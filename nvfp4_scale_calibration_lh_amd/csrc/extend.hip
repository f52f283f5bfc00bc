// Growth of the paged cache's sequences by one step's tokens: block tables, lengths, the stack of free pages
// and, for every new token's row, its slot, position and sequence.
//
// With p tokens a page, request b of length l and n new tokens:
//   n < 0  the last -n tokens leave; the pages that empties go on the stack, in the order of requests and pages
//   n > 0  rows [start_b, start_b + n) are its tokens l .. l + n - 1, for which it needs
//          up((l + n) / p) - up(l / p) pages more; it gets them if the sum of what requests up to it need is
//          at most what the stack then holds (who needs none always goes on), the stack's top first
//
// The work is three sums over the requests (pages given back, rows, pages needed) and one look-up a row.
// One workgroup does the sums: in LDS, with the look-ups after them, where there are few of both; otherwise into
// a workspace, from which a second kernel takes the rows, spread over the chip.  A page that one request
// gives back and another takes in the same step is read from the giver's table, so that neither kernel waits for
// a write to the stack.
//
// Bound by latencies: of a launch, and of a chain of three loads a row (start, table or stack, store).  One token for each of 64
// sequences 4.8 us; 900000 rows of 1024 sequences, 14 MB written, 18.4 us: the sums 7.4, the rows 9.3.
#include "lh_internal.hpp"

#include <algorithm>

namespace lh {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kRun = 256;                    // rows of one workgroup of the second kernel, one a thread (four a thread: 4 us more for 900000)
constexpr int kWindow = 256;                 // sequences whose first rows it holds

struct Args {
  int* table;
  const int* lengths;
  const int* asked;
  int* stack;
  const int* count;
  int64_t* slots;
  int* positions;
  int* sequence;
  int* offsets;
  int* new_lengths;
  int* new_count;
  int* work;
  int64_t width;
  int batch, rows, page, capacity, most;     // most: tokens that a table holds
};

// What the sums leave for the rows: per request (and one past the last) its first row, its length, the pages
// given back before it and its first page that is given back, and the place on the stack of its first new page, or kRefused.
constexpr int kRefused = -2147483647 - 1;
struct Plan {
  int* head;                                 // pages on the stack at first; with those given back; the number of those
  int *start, *len, *freed, *kept, *top;
  __device__ Plan(int* at, int n) : head(at), start(at + 4), len(start + n), freed(len + n), kept(freed + n), top(kept + n) {}
};
constexpr int64_t plan_ints(int64_t batch) { return 4 + 5 * (batch + 1); }

__device__ inline int pages(int tokens, int page) { return (int)(((uint32_t)tokens + (uint32_t)page - 1) / (uint32_t)page); }
__device__ inline int clamp32(int64_t v) { return (int)min(v, (int64_t)2147483647); }

// Inclusive sum over the workgroup; `all` is the whole sum.  Every thread has to come here.
__device__ inline int64_t scan(int64_t v, int64_t* shared, int64_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  if (waves == 1) {
    all = __shfl(v, 63, 64);
    return v;
  }
  __syncthreads();
  if (lane == 63) shared[wave] = v;
  __syncthreads();
  all = 0;
  int64_t before = 0;
  for (int w = 0; w < waves; ++w) {
    before += w < wave ? shared[w] : 0;
    all += shared[w];
  }
  return v + before;
}

__device__ void sums(const Args& a, const Plan& p, int64_t* shared) {
  int64_t freed = 0, rows = 0;
  const int given = *a.count;
  const int count = min(max(given, 0), a.capacity);
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int len = 0, n = 0;
    if (b < a.batch) {
      len = min(max(a.lengths[b], 0), a.most);
      n = a.asked ? a.asked[b] : 1;
    }
    const int cut = (int)max((int64_t)len + min(n, 0), (int64_t)0);
    const int kept = pages(cut, a.page), back = pages(len, a.page) - kept, more = max(n, 0);
    int64_t all_back, all_rows;
    const int64_t upto_back = scan(back, shared, all_back), upto_rows = scan(more, shared, all_rows);
    if (b < a.batch) {
      p.start[b] = (int)min(rows + upto_rows - more, (int64_t)a.rows);
      p.len[b] = len;
      p.freed[b] = clamp32(freed + upto_back - back);
      p.kept[b] = kept;
    }
    freed += all_back;
    rows += all_rows;
  }
  const int avail = (int)min(count + freed, (int64_t)a.capacity);
  if (threadIdx.x == 0) {
    p.start[a.batch] = a.offsets[a.batch] = (int)min(rows, (int64_t)a.rows);
    p.freed[a.batch] = clamp32(freed);
    p.head[0] = count;
    p.head[1] = avail;
    p.head[2] = clamp32(freed);
  }
  int64_t needed = 0;
  int taken = 0;
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int len = 0, n = 0, start = 0;
    if (b < a.batch) {
      len = p.len[b];                         // written by this thread
      start = p.start[b];
      n = a.asked ? a.asked[b] : 1;
    }
    const int more = max(n, 0);
    // a start that was cut to `rows` belongs to a request that has no room either way
    const bool fits = (int64_t)len + more <= a.most && (int64_t)start + more <= a.rows;
    const int need = fits ? pages(len + more, a.page) - pages(len, a.page) : 0;
    int64_t all;
    const int64_t upto = needed + scan(need, shared, all);
    const bool granted = fits && (need == 0 || upto <= avail);
    if (b < a.batch) {
      a.offsets[b] = start;
      p.top[b] = granted ? (int)max(avail - 1 - (upto - need), (int64_t)-1) : kRefused;
      const int cut = (int)max((int64_t)len + min(n, 0), (int64_t)0);
      a.new_lengths[b] = granted ? cut + more : cut;
    }
    if (upto <= avail) taken = max(taken, (int)upto);
    needed += all;
  }
  // the largest over the workgroup
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) taken = max(taken, __shfl_xor(taken, o, 64));
  if (blockDim.x > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = taken;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) taken = max(taken, (int)shared[w]);
  }
  if (threadIdx.x == 0) *a.new_count = avail - taken;
}

// The last of v[lo .. hi] that is at most x; v[lo] is.
__device__ inline int last_upto(const int* v, int x, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The i-th page given back.
__device__ inline int given_back(const Args& a, const Plan& p, int i) {
  const int b = last_upto(p.freed, i, 0, a.batch - 1);
  return a.table[b * a.width + p.kept[b] + (i - p.freed[b])];
}

// Row r of sequence b (the batch's size: behind the last sequence).
__device__ inline void one_row(const Args& a, const Plan& p, int r, int b, int count) {
  int64_t slot = -1;
  int position = -1, sequence = -1;
  if (b < a.batch) {
    sequence = b;
    const int top = p.top[b];
    if (top != kRefused) {
      const int len = p.len[b];
      position = len + (r - p.start[b]);
      const int at = (int)((uint32_t)position / (uint32_t)a.page), off = position - at * a.page, fresh = at - pages(len, a.page);
      int* entry = a.table + b * a.width + at;
      int which;
      if (fresh < 0) {
        which = *entry;
      } else {
        const int place = top - fresh;
        which = place < count ? a.stack[place] : given_back(a, p, place - count);
        if (off == 0) *entry = which;        // of a new page the first token is new
      }
      slot = (int64_t)which * a.page + off;
    }
  }
  a.slots[r] = slot;
  a.positions[r] = position;
  a.sequence[r] = sequence;
}

__global__ __launch_bounds__(kMaxThreads) void k_extend(const Args a) {
  __shared__ int64_t shared[kMaxThreads / 64];
  extern __shared__ int lds[];
  const Plan p(lds, a.batch + 1);
  sums(a, p, shared);
  __syncthreads();
  const int count = p.head[0];
  for (int r = threadIdx.x; r < a.rows; r += blockDim.x) one_row(a, p, r, last_upto(p.start, r, 0, a.batch), count);
  const int back = min(p.head[2], a.capacity - count);
  for (int i = threadIdx.x; i < back; i += blockDim.x) a.stack[count + i] = given_back(a, p, i);
}

__global__ __launch_bounds__(kMaxThreads) void k_extend_sums(const Args a) {
  __shared__ int64_t shared[kMaxThreads / 64];
  sums(a, Plan(a.work, a.batch + 1), shared);
}

// The last of v[0 .. n) that is at most x (v[0] is), for the whole workgroup of 256: 256 places at a time.
__device__ inline int last_upto_together(const int* v, int x, int n, int* shared) {
  int lo = 0, span = n;                      // in [lo, lo + span)
  while (span > 1) {
    const int step = (span + 255) / 256;
    const int64_t at = lo + (int64_t)threadIdx.x * step;
    const uint64_t upto = __ballot(at < lo + (int64_t)span && v[min(at, (int64_t)n - 1)] <= x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = __popcll(upto);
    __syncthreads();
    const int before = shared[0] + shared[1] + shared[2] + shared[3] - 1;
    span = min(step, lo + span - (lo + before * step));
    lo += before * step;
  }
  return lo;
}

// A workgroup finds its first row's sequence, takes the starts of the sequences from there on into LDS, and looks its
// rows up among them (in memory, where a run of rows spans more sequences than that).
__global__ __launch_bounds__(256) void k_extend_rows(const Args a) {
  __shared__ int shared[4];
  __shared__ int starts[kWindow];
  const Plan p(a.work, a.batch + 1);
  const int count = p.head[0], back = min(p.head[2], a.capacity - count);
  const int64_t r0 = (int64_t)blockIdx.x * kRun;
  if (r0 < a.rows) {
    const int r1 = (int)min(r0 + kRun, (int64_t)a.rows);
    const int lo = last_upto_together(p.start, (int)r0, a.batch + 1, shared), held = min(kWindow, a.batch + 1 - lo);
    if ((int)threadIdx.x < held) starts[threadIdx.x] = p.start[lo + threadIdx.x];
    __syncthreads();
    const int r = (int)r0 + threadIdx.x;
    if (r < r1) {
      int b = lo + last_upto(starts, r, 0, held - 1);
      if (b == lo + held - 1 && b < a.batch) b = last_upto(p.start, r, b, a.batch);
      one_row(a, p, r, b, count);
    }
  }
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < back; i += (int64_t)gridDim.x * 256)
    a.stack[count + i] = given_back(a, p, (int)i);
}

// One workgroup: a token for each of 256 and 512 sequences 6.0 and 6.6 us, with two kernels 7.9 and 9.4; 500 tokens of one sequence 5.4 and 6.1.
// More rows than that take it several turns: 1000 tokens of one sequence 7.8 us, 6.1 with two; and so do pages that are given back, where two
// kernels win at any size: a quarter of 200 or 500 sequences of some 8000 tokens ending at once 20 and 25 us, 9.6 and 12 with two.
bool together(int64_t batch, int64_t rows) { return batch <= 512 && rows <= 512; }

}  // namespace

int64_t extend_workspace(int64_t batch, int64_t rows) { return together(batch, rows) ? 0 : 4 * plan_ints(batch); }

hipError_t launch_extend(const ExtendView& v, void* work, hipStream_t stream) {
  Args a{};
  a.table = v.table;
  a.lengths = v.lengths;
  a.asked = v.asked;
  a.stack = v.stack;
  a.count = v.count;
  a.slots = v.slots;
  a.positions = v.positions;
  a.sequence = v.sequence;
  a.offsets = v.offsets;
  a.new_lengths = v.new_lengths;
  a.new_count = v.new_count;
  a.work = (int*)work;
  a.width = v.width;
  a.batch = (int)v.batch;
  a.rows = (int)v.rows;
  a.page = (int)v.page;
  a.capacity = (int)v.capacity;
  a.most = (int)(v.width * v.page);
  auto threads = [](int64_t n) { return dim3((unsigned)std::clamp<int64_t>((n + 63) / 64 * 64, 64, kMaxThreads)); };
  if (together(v.batch, v.rows))
    return launch_kernel(k_extend, dim3(1), threads(std::max(v.batch, v.rows)), (size_t)(4 * plan_ints(v.batch)), stream, a);
  const hipError_t e = launch_kernel(k_extend_sums, dim3(1), threads(v.batch), 0, stream, a);
  if (e != hipSuccess) return e;
  return launch_kernel(k_extend_rows, dim3((unsigned)std::max<int64_t>(64, (v.rows + kRun - 1) / kRun)), dim3(256), 0, stream, a);
}

}  // namespace lh
