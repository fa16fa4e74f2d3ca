// Block tables and slot maps from request lengths: the bookkeeping between two
// steps of a server on a paged cache, on the device, in one launch.
//
//   base_b = seq_b + accept_b + 1   (0 for a finished request)
//   need_b = ceil((base_b + new_b) / P),  ask_b = (need_b - held_b)+,
//   give_b = (held_b - need_b)+
//
// Exclusive prefix sums over the requests place every page and row: request b
// takes entries head + sum_{c<b} ask_c .. of the ring of free pages, gives its
// surplus pages to entries tail + sum_{c<b} give_c .., and its rows start at
// sum_{c<b} new_c.  Every CTA computes the same sums (B <= 4096: at most four
// requests a thread), which needs no exchange between CTAs; then the rows and
// the pages that change hands are spread over all threads of the grid, each
// finding its request by bisection in the sums kept in shared memory.  Pages
// taken are read from the ring and pages kept from the table entries that the
// call does not write, so no thread waits for another's store.
//
// Bound by latency: lengths, then ring and table entries, then stores, 6.3 us in
// a graph for 128 requests of 8 rows (8 us a call from Python; its bytes are
// 10 KB).  2048 prompts with a million rows (17 MB, 2.5 us of copying) take
// 12.3 to 14.3 us: instructions, the rows' bisections of 11 steps each in shared memory
// (16.4 us with divisions by the page size and a loop over the warps' sums).
#include "spec_serve.cuh"

namespace spec {

struct TablesParams {
  int B, P, page_bits, num_pages, stride, max_rows;
  const int* seq_len;
  const int* accept_len;
  const int* new_len;
  const int* num_blocks;
  const long long* ring_pos;
  int* ring;
  int* table;
  int* seq_out;
  int* kv_len;
  int* num_blocks_out;
  long long* ring_pos_out;
  int* row_ptr;
  int* slots;
  int* positions;
  uint32_t* status;
};

constexpr int TABLES_ITEMS = 4;            // requests a thread: 1024 threads x 4 = 4096

struct TablesRequest {
  int base, add, need, held;
};

__device__ __forceinline__ TablesRequest tables_request(const TablesParams& p, int b, bool& bad) {
  const int seq = __ldg(p.seq_len + b), acc = p.accept_len ? __ldg(p.accept_len + b) : -1;
  const int add = __ldg(p.new_len + b), held = __ldg(p.num_blocks + b);
  const long long base = add == -1 ? 0 : (long long)seq + acc + 1;
  const long long kv = base + (add > 0 ? add : 0);
  TablesRequest r;
  r.held = held;
  bad = seq < 0 || acc < -1 || add < -1 || held < 0 || held > p.stride || kv > (long long)p.stride * p.P ||
        kv > 0x3fffffff || ((base + p.P - 1) >> p.page_bits) > held;
  if (bad) {
    r.base = seq;
    r.add = 0;
    r.need = held;
  } else {
    r.base = (int)base;
    r.add = add > 0 ? add : 0;
    r.need = (int)((kv + p.P - 1) >> p.page_bits);
  }
  return r;
}

// Inclusive scans over the CTA of two values a thread; totals over the CTA.
struct Two {
  unsigned long long pages, rows;
};
__device__ __forceinline__ Two warp_scan(Two v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long a = __shfl_up_sync(0xffffffffu, v.pages, o), b = __shfl_up_sync(0xffffffffu, v.rows, o);
    if (lane >= o) {
      v.pages += a;
      v.rows += b;
    }
  }
  return v;
}
__device__ __forceinline__ Two block_scan(Two v, Two* s_warp, Two& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_scan(v, lane);
  __syncthreads();                          // s_warp may still be read from the last scan
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  // every warp scans the warps' sums
  const Two w = warp_scan(lane < nw ? s_warp[lane] : Two{0, 0}, lane);
  const int from = (warp + 31) & 31;
  const Two before{__shfl_sync(0xffffffffu, w.pages, from), __shfl_sync(0xffffffffu, w.rows, from)};
  total = Two{__shfl_sync(0xffffffffu, w.pages, 31), __shfl_sync(0xffffffffu, w.rows, 31)};
  return warp ? Two{v.pages + before.pages, v.rows + before.rows} : v;
}

// Last b in [0, n) with ptr[b] <= x (ptr ascending, ptr[0] <= x).
__device__ __forceinline__ int last_at_or_below(const int* ptr, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ptr[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(1024) block_tables_kernel(TablesParams p) {
  extern __shared__ int s_tab[];            // [5][B + 1]
  __shared__ Two s_warp[32];
  __shared__ int s_first;
  const int B = p.B, n1 = B + 1;
  int* s_row = s_tab;                       // first row of each request
  int* s_ask = s_tab + n1;                  // pages taken before it
  int* s_give = s_tab + 2 * n1;             // pages given before it
  int* s_base = s_tab + 3 * n1;
  int* s_held = s_tab + 4 * n1;
  const int items = (B + blockDim.x - 1) / blockDim.x;
  const int b0 = threadIdx.x * items;

  const long long head = p.ring_pos[0], tail = p.ring_pos[1];
  long long free_pages = tail - head;
  const bool bad_ring = head < 0 || free_pages < 0 || free_pages > p.num_pages;
  if (bad_ring) free_pages = 0;
  const int head_at = bad_ring ? 0 : (int)(head % p.num_pages);
  const int tail_at = bad_ring ? 0 : (int)(tail % p.num_pages);

  TablesRequest r[TABLES_ITEMS];
  uint32_t flags = bad_ring ? SPEC_DEV_BAD_LEN : 0;
  uint32_t badbits = 0;
#pragma unroll
  for (int i = 0; i < TABLES_ITEMS; ++i) {
    r[i] = TablesRequest{0, 0, 0, 0};
    if (i < items && b0 + i < B) {
      bool bad;
      r[i] = tables_request(p, b0 + i, bad);
      if (bad) {
        flags |= SPEC_DEV_BAD_LEN;
        badbits |= 1u << i;
      }
    }
  }
  if (threadIdx.x == 0) s_first = B;

  unsigned long long total_pages, total_rows, pages_at, rows_at;
  for (int pass = 0; pass < 2; ++pass) {
    // pages taken in the low word, pages given in the high word: each total is
    // below 2^31 (B * stride is)
    unsigned long long pages = 0, rows = 0;
#pragma unroll
    for (int i = 0; i < TABLES_ITEMS; ++i) {
      const int d = r[i].need - r[i].held;
      pages += d > 0 ? (unsigned long long)d : (unsigned long long)(-d) << 32;
      rows += (unsigned long long)r[i].add;
    }
    Two all;
    const Two upto = block_scan(Two{pages, rows}, s_warp, all);
    total_pages = all.pages;
    total_rows = all.rows;
    pages_at = upto.pages - pages;
    rows_at = upto.rows - rows;
    const bool fits = (long long)(total_pages & 0xffffffffu) <= free_pages &&
                      total_rows <= (unsigned long long)p.max_rows;
    if (fits || pass) break;                // uniform over the CTA
    // the first request that finds no room; it and every later one append nothing
    unsigned long long a = pages_at & 0xffffffffu, w = rows_at;
#pragma unroll
    for (int i = 0; i < TABLES_ITEMS; ++i) {
      if (i >= items || b0 + i >= B) break;
      const int d = r[i].need - r[i].held;
      a += d > 0 ? d : 0;
      w += r[i].add;
      if (r[i].add > 0 && ((long long)a > free_pages || w > (unsigned long long)p.max_rows)) {
        atomicMin(&s_first, b0 + i);
        break;
      }
    }
    __syncthreads();
    const int first = s_first;
#pragma unroll
    for (int i = 0; i < TABLES_ITEMS; ++i)
      if (i < items && b0 + i < B && b0 + i >= first && r[i].add > 0) {
        r[i].add = 0;
        r[i].need = (int)(((long long)r[i].base + p.P - 1) >> p.page_bits);
        flags |= SPEC_DEV_NO_PAGES;
      }
  }

  // a ring that cannot be, or that has no room for what comes back (a page that
  // is free and held at once: entries to write would be entries that other
  // threads read), takes nothing: requests keep their pages
  const bool over = free_pages + (long long)(total_pages >> 32) > p.num_pages;
  if (over) flags |= SPEC_DEV_BAD_LEN;
  const bool keep = bad_ring || over;
  {
    int ask = (int)(pages_at & 0xffffffffu), give = keep ? 0 : (int)(pages_at >> 32), row = (int)rows_at;
#pragma unroll
    for (int i = 0; i < TABLES_ITEMS; ++i) {
      const int b = b0 + i;
      if (i >= items || b >= B) break;
      if (keep && r[i].need < r[i].held) r[i].need = r[i].held;
      s_row[b] = row;
      s_ask[b] = ask;
      s_give[b] = give;
      s_base[b] = r[i].base;
      s_held[b] = r[i].held;
      if (blockIdx.x == 0) {
        p.seq_out[b] = r[i].base;
        p.kv_len[b] = (badbits >> i) & 1 ? 0 : r[i].base + r[i].add;
        p.num_blocks_out[b] = r[i].need;
        p.row_ptr[b] = row;
      }
      const int d = r[i].need - r[i].held;
      if (d > 0) ask += d; else give -= d;
      row += r[i].add;
    }
  }
  const int n_rows = (int)total_rows, n_ask = (int)(total_pages & 0xffffffffu), n_give = keep ? 0 : (int)(total_pages >> 32);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.row_ptr[B] = n_rows;
    p.ring_pos_out[0] = head + n_ask;
    p.ring_pos_out[1] = tail + n_give;
  }
  if (threadIdx.x == 0) s_row[B] = n_rows;
  __syncthreads();

  const int gid = blockIdx.x * blockDim.x + threadIdx.x, gsz = gridDim.x * blockDim.x;
  // entry of the m-th page taken: m < n_ask <= free pages <= num_pages, so one
  // subtraction is the remainder
  auto taken = [&](int m) {
    const uint32_t at = (uint32_t)head_at + (uint32_t)m;
    return at >= (uint32_t)p.num_pages ? at - (uint32_t)p.num_pages : at;
  };
  // pages that change hands
  for (int m = gid; m < n_ask + n_give; m += gsz) {
    if (m < n_ask) {
      const int b = last_at_or_below(s_ask, B, m);
      p.table[(size_t)b * p.stride + s_held[b] + (m - s_ask[b])] = p.ring[taken(m)];
    } else {
      const int g = m - n_ask, b = last_at_or_below(s_give, B, g);
      const int count = (b + 1 < B ? s_give[b + 1] : n_give) - s_give[b];
      const uint32_t at = ((uint32_t)tail_at + g) % p.num_pages;
      p.ring[at] = p.table[(size_t)b * p.stride + s_held[b] - count + (g - s_give[b])];
    }
  }
  // rows: four consecutive ones a thread
  for (long long r4 = (long long)gid * 4; r4 < p.max_rows; r4 += (long long)gsz * 4) {
    int slot[4], pos[4];
    int b = r4 < n_rows ? last_at_or_below(s_row, B, (int)r4) : 0;
    int last_b = -1, last_blk = 0, page = 0;                 // the page of the row before
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (int)r4 + i;
      slot[i] = pos[i] = -1;
      if (row >= n_rows) continue;
      while (s_row[b + 1] <= row) ++b;
      pos[i] = s_base[b] + row - s_row[b];
      const int blk = pos[i] >> p.page_bits;
      if (b != last_b || blk != last_blk) {
        const int held = s_held[b];
        page = blk < held ? __ldg(p.table + (size_t)b * p.stride + blk) : p.ring[taken(s_ask[b] + blk - held)];
        last_b = b;
        last_blk = blk;
      }
      if (page < 0 || page >= p.num_pages) flags |= SPEC_DEV_BAD_SLOT;
      else slot[i] = (page << p.page_bits) + (pos[i] & (p.P - 1));
    }
    if (r4 + 4 <= p.max_rows) {
      *reinterpret_cast<int4*>(p.slots + r4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + r4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r4 + i < p.max_rows) {
          p.slots[r4 + i] = slot[i];
          p.positions[r4 + i] = pos[i];
        }
    }
  }
  if (flags) set_status(p.status, flags);
}

cudaError_t launch_block_tables(const spec_block_tables_args& a, int sms, cudaStream_t st) {
  TablesParams p{a.B, a.page_size, __builtin_ctz(a.page_size), a.num_pages, a.table_stride, a.max_rows, a.seq_len, a.accept_len, a.new_len,
                 a.num_blocks, (const long long*)a.ring_pos, a.free_ring, a.block_table, a.seq_len_out, a.kv_len,
                 a.num_blocks_out, (long long*)a.ring_pos_out, a.row_ptr, a.slots, a.positions, a.dev_status};
  const int threads = a.B <= 256 ? 256 : 1024;
  long long ctas = ((long long)a.max_rows + 4LL * threads - 1) / (4LL * threads);
  if (ctas < 1) ctas = 1;
  if (ctas > sms) ctas = sms;
  const size_t smem = (size_t)5 * (a.B + 1) * sizeof(int);
  if (smem > 47 * 1024) {                   // 48 KB less the static arrays need no asking
    const cudaError_t e = cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem);
    if (e != cudaSuccess) return e;
  }
  block_tables_kernel<<<(int)ctas, threads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace spec
