// Page operations of the 8-bit cache: lengths, page tables and the copies that go with them.
//
// The bookkeeping of a call is one block of 1024 threads (one thread per list entry, at most
// 1024): it checks the whole list, finds the lowest free pages by a scan of the reference counts
// (so page numbers do not depend on the run), and either changes everything or nothing.  What
// it decided is left in the cache (moves, pairs) for the copying kernels, which are plain
// streams bound by HBM: 16-byte vectors, four in flight per thread, one 16 KB segment of a page
// at a time over all SMs (with the bookkeeping, 0.8 of the measured copy rate over a whole copy
// and compaction).  Launch order on the stream is the only synchronisation.
#include <algorithm>

#include "woq_internal.h"
#include "woq_kv8_device.cuh"

namespace woq {
namespace kv8 {

constexpr int kMetaThreads = 1024;

struct MetaShared {
  int sums[33];
  uint32_t used[kKv8MaxSeqs / 32];
};

// The `need` lowest free pages below `limit` into out; returns how many there are (at most need).
// out may be the map array: only reference counts are read.
__device__ int find_free(const Kv8View& v, int limit, int need, int32_t* out, MetaShared& sh) {
  const int32_t* refs = v.refs_p();
  int found = 0;
  for (int base = 0; base < limit && found < need; base += 4 * kMetaThreads) {
    const int p0 = base + 4 * (int)threadIdx.x;
    int4 r = {1, 1, 1, 1};
    if (p0 + 3 < limit) {
      r = *reinterpret_cast<const int4*>(refs + p0);
    } else {
      if (p0 < limit) r.x = refs[p0];
      if (p0 + 1 < limit) r.y = refs[p0 + 1];
      if (p0 + 2 < limit) r.z = refs[p0 + 2];
    }
    const int f = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int total;
    int rank = found + block_exclusive_sum(f, sh.sums, &total);
    if (r.x == 0 && rank < need) out[rank] = p0;
    rank += r.x == 0;
    if (r.y == 0 && rank < need) out[rank] = p0 + 1;
    rank += r.y == 0;
    if (r.z == 0 && rank < need) out[rank] = p0 + 2;
    rank += r.z == 0;
    if (r.w == 0 && rank < need) out[rank] = p0 + 3;
    found += total;
  }
  __syncthreads();
  return found < need ? found : need;
}

__device__ __forceinline__ void clear_used(MetaShared& sh) {
  if (threadIdx.x < kKv8MaxSeqs / 32) sh.used[threadIdx.x] = 0;
  __syncthreads();
}

// Marks seq; false if it was marked before.
__device__ __forceinline__ bool mark(MetaShared& sh, int seq) {
  const uint32_t bit = 1u << (seq & 31);
  return (atomicOr(&sh.used[seq >> 5], bit) & bit) == 0;
}

__device__ __forceinline__ bool in_range(const Kv8View& v, int seq) { return seq >= 0 && seq < v.seqs; }

__global__ void __launch_bounds__(256) init_kernel(Kv8View v) {
  begin_after_prior();
  if (threadIdx.x == 0) {
    uint32_t* h = v.status();
    h[0] = 0;
    h[2] = v.hash;
    h[3] = (uint32_t)v.pages;
    h[1] = kKv8Magic;
  }
}

__global__ void __launch_bounds__(kMetaThreads) extend_kernel(Kv8View v, int seq, int tokens) {
  __shared__ MetaShared sh;
  begin_after_prior();
  if (!header_ok(v)) return;
  const int len = v.lens_p()[seq];
  bool ok = true;
  if ((long long)len + tokens > v.max_tokens) {
    ok = false;
    if (threadIdx.x == 0) flag(v, WOQ_DEVERR_STATE);
  }
  const int first = len / kKv8Block;
  int need = 0;
  if (ok) {
    need = (len + tokens) / kKv8Block - first;
    if (find_free(v, *v.limit_p(), need, v.map_p(), sh) < need) {
      ok = false;
      if (threadIdx.x == 0) flag(v, WOQ_DEVERR_PAGES);
    }
  }
  __syncthreads();
  if (ok) {
    for (int i = threadIdx.x; i < need; i += kMetaThreads) {
      const int page = v.map_p()[i];
      v.table_row(seq)[first + i] = page;
      v.refs_p()[page] = 1;
    }
  }
  if (threadIdx.x == 0) {
    // Refused: the pending prompt stays, unless it has as many tokens; fills that follow could then be meant for the
    // refused one, and would go over the earlier one's tokens.
    if (ok) v.lens_p()[seq] = len + tokens;
    if (ok) v.reserved_p()[seq] = tokens;
    else if (v.reserved_p()[seq] == tokens) v.reserved_p()[seq] = 0;
  }
}

// moves[e] = {length before, kept rows, page of the block that becomes full or -1, sequence}
__global__ void __launch_bounds__(kMetaThreads)
    accept_meta_kernel(Kv8View v, const int32_t* seqs, int n, const uint32_t* keep) {
  __shared__ MetaShared sh;
  begin_after_prior();
  if (!header_ok(v)) return;
  clear_used(sh);
  const int e = threadIdx.x;
  bool bad = false;
  int seq = 0, len = 0, kept = 0, full = 0;
  uint32_t k = 0;
  if (e < n) {
    seq = seqs ? seqs[e] : e;
    k = keep[e];
    bad = !in_range(v, seq) || k > 0xFFu || !mark(sh, seq);
    if (!bad) {
      len = v.lens_p()[seq];
      kept = __popc(k);
      bad = len + kept > v.max_tokens;
      full = (len % kKv8Block + kept) >= kKv8Block;
    }
  }
  bool ok = true;
  if (__syncthreads_or(bad)) {
    ok = false;
    if (threadIdx.x == 0) flag(v, WOQ_DEVERR_STATE);
  }
  int need = 0, rank = 0;
  if (ok) {
    rank = block_exclusive_sum(full, sh.sums, &need);
    if (find_free(v, *v.limit_p(), need, v.map_p(), sh) < need) {
      ok = false;
      if (threadIdx.x == 0) flag(v, WOQ_DEVERR_PAGES);
    }
  }
  if (e >= n) return;
  if (!ok) {
    v.moves_p()[e] = make_int4(0, 0, -1, 0);
    return;
  }
  int page = -1;
  if (full) {
    page = v.map_p()[rank];
    v.table_row(seq)[len / kKv8Block] = page;
    v.refs_p()[page] = 1;
  }
  v.lens_p()[seq] = len + kept;
  if (kept) v.reserved_p()[seq] = 0;
  v.moves_p()[e] = make_int4(len, (int)k, page, seq);
}

// fork and copy, bookkeeping.  moves[e] = {source, destination, 1 or 0, length}
__device__ __forceinline__ bool check_pairs(const Kv8View& sv, const Kv8View& dv, const int32_t* src,
                                            const int32_t* dst, int n, bool same, MetaShared& sh, int* s, int* d,
                                            int* len) {
  clear_used(sh);
  const int e = threadIdx.x;
  bool bad = false;
  if (e < n) {
    *s = src[e];
    *d = dst[e];
    bad = !in_range(sv, *s) || !in_range(dv, *d) || !mark(sh, *d);
    if (!bad) {
      *len = sv.lens_p()[*s];
      bad = dv.lens_p()[*d] != 0 || *len > dv.max_tokens;
    }
  }
  __syncthreads();
  if (e < n && !bad && same) bad = (sh.used[*s >> 5] >> (*s & 31)) & 1u;
  return !__syncthreads_or(bad);
}

__global__ void __launch_bounds__(kMetaThreads)
    fork_meta_kernel(Kv8View v, const int32_t* src, const int32_t* dst, int n) {
  __shared__ MetaShared sh;
  begin_after_prior();
  if (!header_ok(v)) return;
  int s = 0, d = 0, len = 0;
  const bool ok = check_pairs(v, v, src, dst, n, true, sh, &s, &d, &len);
  if (!ok && threadIdx.x == 0) flag(v, WOQ_DEVERR_STATE);
  const int e = threadIdx.x;
  if (e >= n) return;
  v.moves_p()[e] = make_int4(s, d, ok, len);
  if (ok) {
    v.lens_p()[d] = len;
    v.reserved_p()[d] = 0;
    // a prompt that layers have yet to fill would be filled for the source alone
    v.reserved_p()[s] = 0;
  }
}

__global__ void __launch_bounds__(kMetaThreads)
    copy_meta_kernel(Kv8View sv, Kv8View dv, const int32_t* src, const int32_t* dst, int n, int same) {
  __shared__ MetaShared sh;
  __shared__ int offs[kKv8MaxSeqs + 1];
  begin_after_prior();
  if (!header_ok(dv)) return;
  const uint4 hs = *reinterpret_cast<const uint4*>(sv.base);
  int s = 0, d = 0, len = 0;
  bool ok = hs.y == kKv8Magic && hs.z == sv.hash;
  const int e = threadIdx.x;
  if (!ok) {
    if (threadIdx.x == 0) flag(dv, WOQ_DEVERR_HEADER);
  } else if (!check_pairs(sv, dv, src, dst, n, same, sh, &s, &d, &len)) {
    ok = false;
    if (threadIdx.x == 0) flag(dv, WOQ_DEVERR_STATE);
  }
  int need = 0;
  if (ok) {
    const int mine = e < n ? len / kKv8Block : 0;
    const int at = block_exclusive_sum(mine, sh.sums, &need);
    offs[e] = at;
    if (e == 0) offs[kKv8MaxSeqs] = need;
    if (find_free(dv, *dv.limit_p(), need, dv.map_p(), sh) < need) {
      ok = false;
      if (threadIdx.x == 0) flag(dv, WOQ_DEVERR_PAGES);
    }
  }
  if (e < n) {
    dv.moves_p()[e] = make_int4(s, d, ok, len);
    if (ok) {
      dv.lens_p()[d] = len;
      dv.reserved_p()[d] = 0;
    }
  }
  if (threadIdx.x == 0) dv.pairs_p()[0] = ok ? need : 0;
  __syncthreads();
  if (!ok) return;
  int2* pairs = reinterpret_cast<int2*>(dv.pairs_p()) + 1;
  for (int i = threadIdx.x; i < need; i += kMetaThreads) {
    int lo = 0, hi = n - 1;  // the entry whose range holds i: the last with offs <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (offs[mid] <= i) lo = mid; else hi = mid - 1;
    }
    const int b = i - offs[lo];
    const int page = dv.map_p()[i];
    pairs[i] = make_int2(sv.table_row(src[lo])[b], page);
    dv.table_row(dst[lo])[b] = page;
    dv.refs_p()[page] = 1;
  }
}

__global__ void __launch_bounds__(kMetaThreads) free_kernel(Kv8View v, const int32_t* seqs, int n) {
  __shared__ MetaShared sh;
  begin_after_prior();
  if (!header_ok(v)) return;
  clear_used(sh);
  const int e = threadIdx.x;
  bool bad = false;
  if (e < n) bad = !in_range(v, seqs[e]) || !mark(sh, seqs[e]);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) flag(v, WOQ_DEVERR_STATE);
    return;
  }
  for (int w = threadIdx.x >> 5; w < n; w += kMetaThreads / 32) {  // a warp per sequence
    const int seq = seqs[w];
    const int blocks = v.lens_p()[seq] / kKv8Block;
    for (int b = threadIdx.x & 31; b < blocks; b += 32) atomicSub(&v.refs_p()[v.table_row(seq)[b]], 1);
  }
  __syncthreads();
  if (e < n) {
    v.lens_p()[seqs[e]] = 0;
    v.reserved_p()[seqs[e]] = 0;
  }
}

__global__ void __launch_bounds__(kMetaThreads) compact_meta_kernel(Kv8View v, int limit) {
  __shared__ MetaShared sh;
  begin_after_prior();
  if (!header_ok(v)) return;
  int32_t* refs = v.refs_p();
  int need = 0;
  for (int base = limit; base < v.pages; base += kMetaThreads) {
    const int p = base + (int)threadIdx.x;
    need += __syncthreads_count(p < v.pages && refs[p] != 0);
  }
  // ranks go to map[0 .. need): need <= free pages below limit <= limit, and map[p] below is for p >= limit
  const bool fits = need <= limit && find_free(v, limit, need, v.map_p(), sh) >= need;
  if (threadIdx.x == 0) {
    v.pairs_p()[0] = fits ? need : 0;
    if (fits) *v.limit_p() = limit;
    else flag(v, WOQ_DEVERR_PAGES);
  }
  if (!fits) return;
  int2* pairs = reinterpret_cast<int2*>(v.pairs_p()) + 1;
  int done = 0;
  for (int base = limit; base < v.pages && done < need; base += kMetaThreads) {
    const int p = base + (int)threadIdx.x;
    const int live = p < v.pages && refs[p] != 0;
    int total;
    const int rank = done + block_exclusive_sum(live, sh.sums, &total);
    if (live) {
      const int to = v.map_p()[rank];
      pairs[rank] = make_int2(p, to);
      refs[to] = refs[p];
      refs[p] = 0;
      v.map_p()[p] = to;
    }
    done += total;
  }
}

// Table entries of moved pages after compact_meta_kernel (a page at or above the limit that a
// sequence holds has just been moved).
__global__ void __launch_bounds__(256) remap_kernel(Kv8View v, int limit) {
  begin_after_prior();
  if (!header_ok(v) || v.pairs_p()[0] == 0) return;
  for (int seq = blockIdx.y; seq < v.seqs; seq += gridDim.y) {
    const int blocks = v.lens_p()[seq] / kKv8Block;
    int32_t* row = v.table_row(seq);
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < blocks; b += gridDim.x * blockDim.x)
      if (row[b] >= limit) row[b] = v.map_p()[row[b]];
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4 * kCopyThreads;  // 16-byte vectors of one segment

// Copies the pages of pairs[]: {page of sv, page of dv}.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(Kv8View sv, Kv8View dv) {
  begin_after_prior();
  if (!header_ok(dv)) return;
  const int count = dv.pairs_p()[0];
  const int2* pairs = reinterpret_cast<const int2*>(dv.pairs_p()) + 1;
  const size_t vecs = dv.page_bytes() / 16;
  const long long segs = (long long)((vecs + kCopyVecs - 1) / kCopyVecs);
  for (long long u = blockIdx.x; u < segs * count; u += gridDim.x) {
    const int2 p = pairs[u / segs];
    const size_t at = (size_t)(u % segs) * kCopyVecs + threadIdx.x;
    const uint4* from = reinterpret_cast<const uint4*>(sv.record(p.x, 0, 0));
    uint4* to = reinterpret_cast<uint4*>(dv.record(p.y, 0, 0));
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * kCopyThreads < vecs) x[i] = __ldcs(from + at + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * kCopyThreads < vecs) to[at + i * kCopyThreads] = x[i];
  }
}

// Tails of moves[]: grid (entries, heads, layers).  share: the page-table row of the source too, and
// a reference on each of its pages (fork).
__global__ void __launch_bounds__(256) copy_tails_kernel(Kv8View sv, Kv8View dv, int share) {
  begin_after_prior();
  const int4 m = dv.moves_p()[blockIdx.x];  // beside the header's read
  if (!header_ok(dv) || !m.z) return;
  const uint16_t* from = sv.tail(blockIdx.z, m.x, blockIdx.y);
  uint16_t* to = dv.tail(blockIdx.z, m.y, blockIdx.y);
  // the tokens and the draft rows behind them: so many rows of keys, and octets of the values' rows
  const int D = dv.dim, rows = m.w % kKv8Block + WOQ_KV8_ROWS, octets = (rows + 7) / 8;
#pragma unroll 4
  for (int i = threadIdx.x; i < rows * (D / 8); i += blockDim.x)
    reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(from)[i];
#pragma unroll 4
  for (int i = threadIdx.x; i < octets * D; i += blockDim.x) {
    const int at = kKv8Tail * D + (i / octets) * kKv8Tail + (i % octets) * 8;
    *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(from + at);
  }
  if (share && blockIdx.y == 0 && blockIdx.z == 0) {
    for (int b = threadIdx.x; b < m.w / kKv8Block; b += blockDim.x) {
      const int page = sv.table_row(m.x)[b];
      dv.table_row(m.y)[b] = page;
      atomicAdd(&dv.refs_p()[page], 1);
    }
  }
}

// One (block of 64 tokens, head, layer) back to bf16.  Bound by HBM: one byte read and two written
// per value.  Keys: a thread's 16 codes are 16 elements of one token.  Values lie transposed, so
// they pass through shared memory: a thread takes four tokens of eight elements (eight words),
// and its four 16-byte rows; cores are spaced 132 bytes apart, which spreads the eight-element
// groups over the banks.
template <int FMT>
__device__ void read_record(const Kv8View& v, const uint8_t* rec, uint32_t* smem, int t0, int t1, uint16_t* k,
                            uint16_t* vals, size_t row, int block_first) {
  const int D = v.dim, chunks = 64 * D / 16;
  const float ks = *reinterpret_cast<const float*>(rec + 128 * (size_t)D);
  const float vs = *reinterpret_cast<const float*>(rec + 128 * (size_t)D + 4);
  const uint4* kc = reinterpret_cast<const uint4*>(rec);
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    const uint4 w = kc[chunks + c];
    const int at = (c >> 3) * 33 + (c & 7) * 4;
    smem[at] = w.x;
    smem[at + 1] = w.y;
    smem[at + 2] = w.z;
    smem[at + 3] = w.w;
  }
  auto two = [&](uint32_t codes, float s) {
    const uint32_t h = f16x2_of_codes<FMT>(codes);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16(f.x * s, f.y * s);
  };
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    const int core = c >> 3, p = (core / (D / 16)) * 8 + (c & 7), d = (core % (D / 16)) * 16;
    const int tok = block_first + kv8_token_of_row(p);
    if (tok < t0 || tok >= t1) continue;
    const uint4 w = kc[c];
    uint4* out = reinterpret_cast<uint4*>(k + (size_t)(tok - t0) * row + d);
    out[0] = make_uint4(two(w.x, ks), two(w.x >> 16, ks), two(w.y, ks), two(w.y >> 16, ks));
    out[1] = make_uint4(two(w.z, ks), two(w.z >> 16, ks), two(w.w, ks), two(w.w >> 16, ks));
  }
  __syncthreads();
  const int groups = D / 8;
  for (int u = threadIdx.x; u < 16 * groups; u += blockDim.x) {
    const int db = u % groups, quad = u / groups;  // four tokens from 4 quad on
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = smem[(db * 4 + (quad >> 2)) * 33 + j * 4 + (quad & 3)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = block_first + 4 * quad + i;
      if (tok < t0 || tok >= t1) continue;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = two(((w[2 * j] >> (8 * i)) & 0xFFu) | (((w[2 * j + 1] >> (8 * i)) & 0xFFu) << 8), vs);
      *reinterpret_cast<uint4*>(vals + (size_t)(tok - t0) * row + db * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

__global__ void __launch_bounds__(256)
    read_kernel(Kv8View v, int layer, int seq, int first, int count, uint16_t* k, uint16_t* vals) {
  __shared__ uint32_t smem[64 * 256 / 128 * 33];
  begin_after_prior();
  // length and page beside the header's read (a row of the table is all there, though only its first entries are set)
  const int b = first / kKv8Block + (int)blockIdx.x;
  const int len = v.lens_p()[seq], page = b < v.blocks ? v.table_row(seq)[b] : 0;
  if (!header_ok(v)) return;
  if ((long long)first + count > (long long)len + WOQ_KV8_ROWS) {
    if (threadIdx.x == 0) flag(v, WOQ_DEVERR_STATE);
    return;
  }
  const int D = v.dim, head = blockIdx.y, full = len / kKv8Block;
  const size_t row = (size_t)v.heads * D;
  k += ((size_t)blockIdx.z * count * v.heads + head) * D;
  vals += ((size_t)blockIdx.z * count * v.heads + head) * D;
  const int l = layer + (int)blockIdx.z;
  if (b < full) {
    const uint8_t* rec = v.record(page, l, head);
    if (v.fmt == WOQ_KV8_INT8) read_record<WOQ_KV8_INT8>(v, rec, smem, first, first + count, k, vals, row, b * kKv8Block);
    else read_record<WOQ_KV8_E4M3>(v, rec, smem, first, first + count, k, vals, row, b * kKv8Block);
    return;
  }
  const uint16_t* tail = v.tail(l, seq, head);
  const int t0 = b * kKv8Block > first ? b * kKv8Block : first;
  const int t1 = (b + 1) * kKv8Block < first + count ? (b + 1) * kKv8Block : first + count;
  const int shift = full * kKv8Block;  // tail rows are token - shift, below 72 (checked above)
#pragma unroll 2
  for (int u = threadIdx.x; u < (t1 - t0) * (D / 8); u += blockDim.x) {
    const int tok = t0 + u / (D / 8), d = (u % (D / 8)) * 8;
    *reinterpret_cast<uint4*>(k + (size_t)(tok - first) * row + d) =
        *reinterpret_cast<const uint4*>(tail + (size_t)(tok - shift) * D + d);
  }
  // values: eight tokens of two elements, then a pair for each token
  const int o0 = (t0 - shift) / 8, octets = (t1 - shift + 7) / 8 - o0;
  const uint16_t* tv = tail + (size_t)kKv8Tail * D;
#pragma unroll 2
  for (int u = threadIdx.x; u < octets * (D / 2); u += blockDim.x) {
    const int d = (u % (D / 2)) * 2, r = (o0 + u / (D / 2)) * 8;
    const uint4 a = *reinterpret_cast<const uint4*>(tv + (size_t)d * kKv8Tail + r);
    const uint4 b = *reinterpret_cast<const uint4*>(tv + (size_t)(d + 1) * kKv8Tail + r);
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int tok = shift + r + i;
      if (tok >= t0 && tok < t1)
        *reinterpret_cast<uint32_t*>(vals + (size_t)(tok - first) * row + d) =
            __byte_perm(x[i >> 1], y[i >> 1], (i & 1) ? 0x7632 : 0x5410);
    }
  }
}

// Words of the bookkeeping to the caller (whose buffer may begin at any word); all threads of the grid.
__device__ __forceinline__ void copy_words(int32_t* to, const int32_t* from, size_t n) {
  if (!to) return;
  const size_t step = (size_t)gridDim.x * blockDim.x;
#pragma unroll 4
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) to[i] = from[i];
}

__global__ void __launch_bounds__(256) state_kernel(Kv8View v, int32_t* lens, int32_t* refs, int32_t* table) {
  begin_after_prior();
  if (!header_ok(v)) return;
  copy_words(lens, v.lens_p(), (size_t)v.seqs);
  copy_words(refs, v.refs_p(), (size_t)v.pages);
  copy_words(table, v.table_row(0), (size_t)v.seqs * v.blocks);
}

}  // namespace kv8

cudaError_t launch_kv8_init(const Kv8View& v, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(v.base, 0, v.pool, s);
  if (e != cudaSuccess) return e;
  return kv8::launch(kv8::init_kernel, 1, 32, 0, s, v);
}

cudaError_t launch_kv8_extend(const Kv8View& v, int seq, int tokens, cudaStream_t s) {
  return kv8::launch(kv8::extend_kernel, 1, kv8::kMetaThreads, 0, s, v, seq, tokens);
}

cudaError_t launch_kv8_accept_meta(const Kv8View& v, const int32_t* seqs, int n, const uint32_t* keep, cudaStream_t s) {
  return kv8::launch(kv8::accept_meta_kernel, 1, kv8::kMetaThreads, 0, s, v, seqs, n, keep);
}

cudaError_t launch_kv8_free(const Kv8View& v, const int32_t* seqs, int n, cudaStream_t s) {
  return kv8::launch(kv8::free_kernel, 1, kv8::kMetaThreads, 0, s, v, seqs, n);
}

static dim3 per_tail(const Kv8View& v, int n) { return dim3((unsigned)n, (unsigned)v.heads, (unsigned)v.layers); }

static cudaError_t copy_pages(const Kv8View& src, const Kv8View& dst, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  return kv8::launch(kv8::copy_pages_kernel, 8 * sms, kv8::kCopyThreads, 0, s, src, dst);
}

cudaError_t launch_kv8_fork(const Kv8View& v, const int32_t* src, const int32_t* dst, int n, cudaStream_t s) {
  const cudaError_t e = kv8::launch(kv8::fork_meta_kernel, 1, kv8::kMetaThreads, 0, s, v, src, dst, n);
  return e != cudaSuccess ? e : kv8::launch(kv8::copy_tails_kernel, per_tail(v, n), 256, 0, s, v, v, 1);
}

cudaError_t launch_kv8_copy(const Kv8View& src, const Kv8View& dst, const int32_t* src_seqs, const int32_t* dst_seqs,
                            int n, cudaStream_t s) {
  const int same = src.base == dst.base;
  cudaError_t e = kv8::launch(kv8::copy_meta_kernel, 1, kv8::kMetaThreads, 0, s, src, dst, src_seqs, dst_seqs, n, same);
  if (e == cudaSuccess) e = kv8::launch(kv8::copy_tails_kernel, per_tail(dst, n), 256, 0, s, src, dst, 0);
  return e != cudaSuccess ? e : copy_pages(src, dst, s);
}

cudaError_t launch_kv8_compact(const Kv8View& v, int limit, cudaStream_t s) {
  cudaError_t e = kv8::launch(kv8::compact_meta_kernel, 1, kv8::kMetaThreads, 0, s, v, limit);
  const dim3 grid(8, (unsigned)(v.seqs < 256 ? v.seqs : 256));
  if (e == cudaSuccess) e = kv8::launch(kv8::remap_kernel, grid, 256, 0, s, v, limit);
  return e != cudaSuccess ? e : copy_pages(v, v, s);
}

cudaError_t launch_kv8_state(const Kv8View& v, int32_t* lens, int32_t* refs, int32_t* table, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  size_t words = 1;
  if (lens) words = std::max(words, (size_t)v.seqs);
  if (refs) words = std::max(words, (size_t)v.pages);
  if (table) words = std::max(words, (size_t)v.seqs * v.blocks);
  const size_t blocks = std::min((words + 4 * 256 - 1) / (4 * 256), (size_t)8 * sms);
  return kv8::launch(kv8::state_kernel, (unsigned)blocks, 256, 0, s, v, lens, refs, table);
}

cudaError_t launch_kv8_read(const Kv8View& v, int layer, int layers, int seq, int first, int count, uint16_t* k,
                            uint16_t* vals, cudaStream_t s) {
  const int blocks = (first + count - 1) / kKv8Block - first / kKv8Block + 1;
  const dim3 grid((unsigned)blocks, (unsigned)v.heads, (unsigned)layers);
  return kv8::launch(kv8::read_kernel, grid, 256, 0, s, v, layer, seq, first, count, k, vals);
}

}  // namespace woq
