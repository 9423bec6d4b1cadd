// pages.cu -- paged-cache bookkeeping around the verification calls (sm_100a): block tables and
// slot maps from request lengths (etree_page_plan), and the store of new K/V rows through a slot
// map (etree_kv_store).
//
// The engines the pages plug into hold KV in pages under continuous batching ("EAGLE-4
// 官方推理代码发布 ...", section on the harness being a plug-in for SGLang and vLLM), and every
// sequence grows by its own accepted length each step ("Eagle-4 Released ...", section "Current
// Limitation"), so the pages of a step are known only on the device.
#include <algorithm>

#include "kernels.cuh"

namespace etree {

// Page plan.  With P tokens a page, request r needs need = ceil((kv + new) / P) pages and holds
// `held`: it takes grow = max(0, need - held) ids from the head of the free ring or gives back
// held - need ids to its tail.  Offsets into the ring are prefix sums over the requests, so the
// result does not depend on any order of execution.
//
// The whole plan is one launch, because its cost is latency: a few dependent reads and one write
// per slot.  Every CTA therefore repeats the prefix sums over all
// B requests (at most 4096, from L2) in shared memory and then takes its share of one flat list
// of work: the pages taken, the pages given back, and the tokens' slots.  Nothing that one CTA
// reads is written by another: table entries below `held` and at or above it are read and written
// apart, the ring's free part and the places behind its tail are disjoint, and the other outputs
// are buffers of their own.  A token's page comes from the ring directly when its table entry is
// being written by this same launch.
constexpr int kPlanThreads = 256;

struct PlanScan {
  long long warp_g[kPlanThreads / 32], warp_r[kPlanThreads / 32], warp_a[kPlanThreads / 32];
  long long taken, back, head, tail;
  int decreasing;                             // cu_new is: a search by halves does not find every token
};

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanParams p) {
  extern __shared__ int32_t plan_s[];
  __shared__ PlanScan sc;
  int32_t* cu_s = plan_s;                     // [B + 1]
  int32_t* kv_s = cu_s + p.B + 1;             // [B]  cached tokens, -1: no slots for this request
  int32_t* held_s = kv_s + p.B;               // [B]  pages held before
  int32_t* need_s = held_s + p.B;             // [B]  pages held after
  int32_t* gend_s = need_s + p.B;             // [B]  inclusive prefix of pages taken (saturated)
  int32_t* rend_s = gend_s + p.B;             // [B]  inclusive prefix of pages given back
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.B;
  const long long cap = p.num_pages;
  for (int i = tid; i <= B; i += kPlanThreads) cu_s[i] = p.cu_new[i];
  for (int i = tid; i < B; i += kPlanThreads) {
    kv_s[i] = p.kv_len[i];
    held_s[i] = p.held[i];
  }
  if (tid == 0) {
    sc.head = p.ring_state[0];
    sc.tail = p.ring_state[1];
    sc.decreasing = 0;
  }
  __syncthreads();
  const long long head = sc.head, tail = sc.tail;
  const bool ring_ok = head >= 0 && tail >= head && tail - head <= cap;
  const long long avail = ring_ok ? tail - head : 0;

  // each thread owns `per` consecutive requests
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(B, tid * per), r1 = min(B, r0 + per);
  long long g = 0, b = 0;
  int bad = 0;                                // a detail code of this thread's requests
  for (int r = r0; r < r1; ++r) {
    const long long n = (long long)cu_s[r + 1] - cu_s[r];
    const long long len = (long long)kv_s[r] + n;
    const int held = held_s[r];
    int code = 0;
    if (n < 0) sc.decreasing = 1;
    if (n < 0 || cu_s[r] < 0 || (p.slot_map && cu_s[r + 1] > p.n_tokens) || (r == 0 && cu_s[0] != 0))
      code = DET_BAD_NODES;
    else if (kv_s[r] < 0 || held < 0 || held > p.max_pages ||
             len > ((long long)p.max_pages << p.page_shift))
      code = DET_KV_LEN;
    if (code) {
      bad = bad ? bad : code;
      kv_s[r] = -1;
      need_s[r] = held;                       // left as it is
    } else {
      const int need = (int)((len + (1ll << p.page_shift) - 1) >> p.page_shift);
      need_s[r] = need;
      g += max(0, need - held);
      b += max(0, held - need);
    }
  }
  // inclusive scan of both sums over the block
  long long gi = g, bi = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long gx = __shfl_up_sync(0xffffffffu, gi, off);
    const long long bx = __shfl_up_sync(0xffffffffu, bi, off);
    if (lane >= off) {
      gi += gx;
      bi += bx;
    }
  }
  if (lane == 31) {
    sc.warp_g[warp] = gi;
    sc.warp_r[warp] = bi;
  }
  __syncthreads();
  long long gp = 0, bp = 0, btot = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) {
      gp += sc.warp_g[w];
      bp += sc.warp_r[w];
    }
    btot += sc.warp_r[w];
  }
  // pages can come back only where the ring has room: more would mean a page counted twice
  const bool back_ok = ring_ok && avail + btot <= cap;
  long long gx = gp + gi - g, bx = bp + bi - b, mine = 0;   // exclusive prefixes
  bool short_of = false;
  for (int r = r0; r < r1; ++r) {
    const int held = held_s[r];
    int need = need_s[r];
    if (need > held) {
      gx += need - held;
      if (gx > avail) {                       // not served, like every later request that grows
        short_of = true;
        need_s[r] = held;
        kv_s[r] = -1;
      }
    } else if (need < held) {
      if (back_ok) bx += held - need;
      else need_s[r] = held;
    }
    if (gx <= avail) mine = gx;
    gend_s[r] = (int32_t)min(gx, (long long)INT32_MAX);
    rend_s[r] = (int32_t)bx;                  // at most `cap`, below 2^31
  }
  // the pages taken: the largest prefix that is served
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, off));
  if (lane == 0) sc.warp_a[warp] = mine;
  const int any_short = __syncthreads_or(short_of);
  long long taken = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) taken = max(taken, sc.warp_a[w]);
  const long long back = back_ok ? btot : 0;
  if (blockIdx.x == 0) {
    if (bad) report(p.ws, ETREE_EDEVICE, bad);
    if (tid == 0) {
      if (!ring_ok || !back_ok) report(p.ws, ETREE_EDEVICE, DET_FREE_RING);
      if (any_short) report(p.ws, ETREE_ENOSPACE, DET_CAPACITY);
      p.ring_state_out[0] = head + taken;
      p.ring_state_out[1] = tail + back;
    }
  }
  const int stride = gridDim.x * kPlanThreads;
  const int i0 = blockIdx.x * kPlanThreads + tid;
  const int P = 1 << p.page_shift;
  for (int r = i0; r < B; r += stride) {
    p.held_out[r] = need_s[r];
    if (p.slot_cap) p.slot_cap[r] = min(max(need_s[r], 0), p.max_pages) << p.page_shift;
  }
  // first request whose inclusive prefix is above i
  auto find = [&](const int32_t* ends, int i) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > i) hi = mid; else lo = mid + 1;
    }
    return lo;
  };
  // 32-bit ring positions: head % cap and an offset, each below 2^31
  const uint32_t ucap = (uint32_t)cap;
  const uint32_t h0 = ring_ok ? (uint32_t)(head % cap) : 0, t0 = ring_ok ? (uint32_t)(tail % cap) : 0;
  auto wrap = [&](uint32_t at) { return at >= ucap ? at - ucap : at; };
  for (long long i = i0; i < taken; i += stride) {
    const int r = find(gend_s, (int)i);
    const int page = need_s[r] - (gend_s[r] - (int)i);
    p.block_table[(size_t)r * p.max_pages + page] = p.ring[wrap(h0 + (uint32_t)i)];
  }
  for (long long i = i0; i < back; i += stride) {
    const int r = find(rend_s, (int)i);
    const int page = held_s[r] - (rend_s[r] - (int)i);
    p.ring[wrap(t0 + (uint32_t)i)] = p.block_table[(size_t)r * p.max_pages + page];
  }
  if (!p.slot_map) return;
  for (long long i = i0; i < p.n_tokens; i += stride) {
    const int j = (int)i;
    long long slot = -1;
    int r;
    if (!sc.decreasing) {
      r = find(cu_s + 1, j);
    } else {                                  // the first valid range that holds the token
      for (r = 0; r < B - 1; ++r)
        if (j >= cu_s[r] && j < cu_s[r + 1] && cu_s[r] >= 0 && cu_s[r + 1] <= p.n_tokens &&
            (r > 0 || cu_s[0] == 0))
          break;
    }
    const int kv = kv_s[r];
    if (kv >= 0 && j >= cu_s[r] && j < cu_s[r + 1]) {
      const int t = kv + (j - cu_s[r]);
      const int pi = t >> p.page_shift;
      const int32_t page =
          pi < held_s[r]
              ? p.block_table[(size_t)r * p.max_pages + pi]
              : p.ring[wrap(h0 + (uint32_t)(gend_s[r] - (need_s[r] - pi)))];
      if (page >= 0 && page < cap)
        slot = ((long long)page << p.page_shift) + (t & (P - 1));
      else
        report(p.ws, ETREE_EDEVICE, DET_BAD_PAGE);
    }
    p.slot_map[i] = slot;
  }
}

cudaError_t launch_page_plan(const PlanParams& p, int sms, cudaStream_t s) {
  const size_t smem = ((size_t)6 * p.B + 1) * sizeof(int32_t);
  if (smem > 40 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(((size_t)6 * ETREE_MAX_REQUESTS + 1) * 4));
    if (e != cudaSuccess) return e;
  }
  const int64_t items = std::max<int64_t>(p.slot_map ? p.n_tokens : 0, (int64_t)p.B * 8);
  const int64_t want = (items + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
  const int grid = (int)std::min<int64_t>(std::max<int64_t>(want, 1), 2 * sms);
  return launch_pdl(page_plan_kernel, dim3(grid), dim3(kPlanThreads), smem, s, p);
}

// K/V store.  A bit copy bound by HBM: every byte is read once and written once.  One warp moves
// the K and the V row of one (token, KV head): lanes 0-15 the 256 bytes of K, lanes 16-31 those of
// V, kStoreUnroll such pairs with all loads in flight before their stores.
constexpr int kStoreThreads = 256;
constexpr int kStoreUnroll = 4;

__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(StoreParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long warp = ((long long)blockIdx.x * kStoreThreads + threadIdx.x) >> 5;
  const long long units = (long long)p.n_tokens * p.hkv;
  const long long u0 = warp * kStoreUnroll;
  if (u0 >= units) return;
  const bool isv = lane >= 16;
  const int col = lane & 15;
  const uint4* src = isv ? p.v : p.k;
  uint4* dst = isv ? p.v_pool : p.k_pool;
  const long long stride = isv ? p.v_stride16 : p.k_stride16;
  int token = (int)(u0 / p.hkv), h = (int)(u0 - (long long)token * p.hkv);
  uint4 v[kStoreUnroll];
  long long to[kStoreUnroll];
#pragma unroll
  for (int i = 0; i < kStoreUnroll; ++i) {
    to[i] = -1;
    if (u0 + i < units) {
      const long long slot = __ldg(p.slot_map + token);
      if (slot >= 0 && slot < p.num_slots) {
        v[i] = __ldg(src + token * stride + h * 16 + col);
        to[i] = (slot * p.hkv + h) * 16 + col;
      } else if (slot != -1 && lane == 0) {
        report(p.ws, ETREE_EDEVICE, DET_BAD_SLOT);
      }
      if (++h == p.hkv) {
        h = 0;
        ++token;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kStoreUnroll; ++i)
    if (to[i] >= 0) dst[to[i]] = v[i];
}

cudaError_t launch_kv_store(const StoreParams& p, cudaStream_t s) {
  const long long units = (long long)p.n_tokens * p.hkv;
  const long long per_cta = (long long)kStoreUnroll * (kStoreThreads / 32);
  const long long grid = (units + per_cta - 1) / per_cta;
  return launch_pdl(kv_store_kernel, dim3((unsigned)grid), dim3(kStoreThreads), 0, s, p);
}

}  // namespace etree
