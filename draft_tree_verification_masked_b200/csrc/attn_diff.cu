// attn_diff.cu -- differential tree attention on tcgen05 / TMEM (sm_100a).
//
// Every tree node attends to its request's cached keys, its tree ancestors and itself, in one
// forward over the whole tree ("Eagle-4 Released: Outpaces DFlash2 and DSpark ...", section
// "Technical Background").  A 128-dim query or key head holds two 64-dim halves, each with a
// softmax map of its own over the same 128-dim values, and the output is their difference:
//
//   a_m = softmax(scale q_m k_m^T), m = 1, 2;   d = a_1 V - lambda_h a_2 V;
//   out = out_scale * d * rsqrt(mean(d^2) + eps) * w        (d * out_scale without w).
//
// Heads and caches have the ordinary attention's layout, and so do its reads: each K/V byte comes
// from HBM once for both maps, all nodes and all query heads of a KV head.  Per 64-key tile:
//
//   S_m  = Q_m K_m^T   tcgen05.mma M=128 (rows) x N=64 (keys) x K=64, the two 64-dim boxes of Q and
//                      K that the TMA loads bring anyway;
//   O_m += P_m V       tcgen05.mma M=128 x N=128 x K=64 for each part of P_m (bf16, from TMEM).
//
// One CTA = (request, KV head, 128-row block, KV split); row = node * G + g.  Warp 0 streams Q and
// the K/V ring; each map has an MMA warp and four softmax warps (one row per thread, one TMEM
// lane).  TMEM holds both O accumulators (256 columns) and two buffers of 64 columns a map, in which
// P's two parts replace the S that they were made from: all 512 columns, so one CTA runs per SM.
// S of tile j + 2 is issued once the products with P of tile j have left its buffer, so S of the
// next tile is always there when the softmax asks for it.
//
// P enters the product with V as the sum of two bf16 operands, off by at most 2^-14 of each value:
// rounding P to one bf16 would add as much to an output's error as its own rounding to bf16 does.
// The row sums add the unrounded fp32 values, and maxima, sums and both outputs stay in fp32 until
// the one rounding of `out`.  O is rescaled only when a row's maximum grows by more than 2^8.
//
// Floor of 64 ragged requests (16 nodes, 40 query heads, 8 KV heads, 1K to 8K cached): 1.23 GB of
// cache, 190 us at the copy rate.  Measured 358 us after a rest, at 1,965 MHz (3.4 TB/s), and 415 us
// in a loop, which meets the power limit at about 1,600 MHz; 128K cached tokens of one request 166
// and 187 us (floor 83); one request with 64 nodes over 4K 33 us (floor 5).  What bounds it is the
// softmax of a tile, instruction by instruction: about 1 us from one S to the next.  Best of eight
// runs, P rounded to one bf16 took 274 us on the ragged batch where two parts took 331, 125 to 130
// against 158 on the long cache and 30 against 32 on the 64 nodes.  Measured with one bf16 P in the
// same way and not kept: sixteen softmax warps with 32 keys each 291 us, the two maps' exponentials
// taking turns 287 us, half of the exponentials as polynomials on the FMA units 331 us.
//
// A key that no row may see takes no part: V rows behind the last cached key and behind the last
// tree node are zeroed in shared memory (0 x NaN would be NaN), and a tree node's infinite or NaN
// values, which only its descendants may see, are taken out of the tile and added to those rows'
// outputs at the end.
#include "kernels.cuh"

namespace etree {

namespace {
constexpr int kDKeys = 64;
constexpr int kDStages = 5;
constexpr int kDBox = kDKeys * 128;         // one [64 keys][64 dims] bf16 box
constexpr int kDKV = 4 * kDBox;             // K halves, V halves
constexpr int kDQ = 2 * 16384;              // Q halves, [128 rows][64 dims]
constexpr float kDLazy = 8.0f;              // rescale O only when the maximum grows by > 2^8
// TMEM columns: O_m at 128 m; buffer b of map m at 256 + 128 m + 64 b: S (fp32), then P's
// parts (32 columns each) in its place
constexpr int kDS = 256, kDCols = 512;
constexpr int kDThreads = 32 * 12;

struct DiffSmem {
  uint64_t kv_full[kDStages], kv_empty[kDStages], q_full, drain[2];
  uint64_t s_full[2][2], p_full[2][2], o_done[2];
  uint64_t o_final[2];                      // the last product of a map is done
  uint64_t v_clean[2];                      // V of the cache's last tile, and of the tree's
  uint64_t anc[64];
  unsigned long long bad;                   // tree nodes whose V holds an infinity or NaN
  int32_t par[64];
  float l[2][128], sq[2][128];              // per map: row sum; per half: sum of d^2
  uint32_t tmem;
};

// Node ranges and lengths that the declared sizes hold.
__device__ __forceinline__ bool diff_nodes_ok(const DiffParams& p, int base, int n) {
  return n >= 1 && n <= p.n_max && base >= 0 && base <= p.n_total - n;
}

__device__ __forceinline__ bool diff_valid(const DiffParams& p, int base, int n, int L,
                                           int64_t sbase) {
  const bool paged = p.block_table != nullptr;
  return diff_nodes_ok(p, base, n) && L >= 0 && L <= p.kv_len_max &&
         (paged || (sbase >= 0 && sbase + L <= p.cache_slots)) &&
         (!paged || L <= ((int64_t)p.max_pages << p.page_shift));
}

__device__ __forceinline__ float bf16_bits(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ bool bf16_nonfinite(uint32_t u) { return (u & 0x7f80u) == 0x7f80u; }

// a w0 + b w1, both products rounded alike (no fused multiply-add), so that equal maps cancel.
__device__ __forceinline__ float diff2(float a, float w0, float b, float w1) {
  return __fadd_rn(__fmul_rn(a, w0), __fmul_rn(b, w1));
}

// A pair of non-negative fp32 values as two pairs of bf16 whose sum is off by at most 2^-14 of the
// value: the upper halves of the words, and what they leave, cut to bf16 as well.
__device__ __forceinline__ uint32_t upper_pair(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ uint32_t lower_pair(float a, float b) {
  float r0 = __uint_as_float((__float_as_uint(a) & 0xffff0000u) | 0x80000000u);   // minus the upper half
  float r1 = __uint_as_float((__float_as_uint(b) & 0xffff0000u) | 0x80000000u);
  fadd2(r0, r1, a, b);
  return upper_pair(r0, r1);
}

// 64 consecutive fp32 columns of this thread's TMEM lane, in one load.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]),
        "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]),
        "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// Writes 16 consecutive 32-bit columns of this thread's TMEM lane without waiting for them.
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void softmax_warps_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}
}  // namespace

__global__ void __launch_bounds__(kDThreads, 1)
attn_diff_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kc,
                 const __grid_constant__ CUtensorMap tm_vc,
                 const __grid_constant__ CUtensorMap tm_kt,
                 const __grid_constant__ CUtensorMap tm_vt, DiffParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + kDQ;
  DiffSmem* sh = reinterpret_cast<DiffSmem*>(sKV + kDStages * kDKV);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_req = p.hkv * p.mchunks;
  const int r = p.order ? p.order[blockIdx.x / per_req] : blockIdx.x / per_req;
  const int kvh = (blockIdx.x % per_req) / p.mchunks;
  const int mb = blockIdx.x % p.mchunks;
  const int s = blockIdx.y;
  const int G = p.G;

  const int base = p.cu_nodes[r];
  const int n = p.cu_nodes[r + 1] - base;
  const int L = p.kv_len[r];
  const bool paged = p.block_table != nullptr;
  const int64_t sbase = paged ? 0 : p.slot_base[r];
  if (!diff_valid(p, base, n, L, sbase)) {
    if (threadIdx.x == 0 && s == 0 && mb == 0 && kvh == 0)
      report(p.ws, ETREE_EDEVICE, diff_nodes_ok(p, base, n) ? DET_KV_LEN : DET_BAD_NODES);
    return;
  }
  const int node0 = mb * p.nb;
  if (node0 >= n) return;
  const int nt_cache = (L + kDKeys - 1) / kDKeys;
  const int total = nt_cache + 1;                       // the tree is the last tile (n <= 64)
  const int t0 = s * p.tps;
  const int t1 = min(total, t0 + p.tps);
  if (t0 >= t1) return;
  const int T = t1 - t0;
  const bool has_tree = t1 == total;
  const int qrows = p.nb * G;                           // rows the Q box fills

  if (threadIdx.x == 0) {
    for (int i = 0; i < kDStages; ++i) {
      mbar_init(&sh->kv_full[i], 1);
      mbar_init(&sh->kv_empty[i], 2);
    }
    mbar_init(&sh->q_full, 1);
    for (int m = 0; m < 2; ++m) {
      mbar_init(&sh->v_clean[m], 8);
      mbar_init(&sh->o_done[m], 1);
      mbar_init(&sh->o_final[m], 1);
      mbar_init(&sh->drain[m], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sh->s_full[m][b], 1);
        mbar_init(&sh->p_full[m][b], 4);
      }
    }
    sh->bad = 0ull;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem, kDCols);
    tmem_relinquish();
  }
  if (has_tree) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) sh->par[i] = p.parent[base + i];
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      uint64_t m = 0;
      int j = i, steps = 0;
      bool ok = true;
      while (j >= 0 && steps <= 64) {
        m |= 1ull << j;
        const int pj = sh->par[j];
        if ((j == 0 && pj != -1) || (j > 0 && (pj < 0 || pj >= j))) { ok = false; break; }
        j = pj;
        ++steps;
      }
      if (!ok) {
        m = 1ull << i;                                  // a malformed tree: each node sees itself
        report(p.ws, ETREE_EDEVICE, DET_BAD_PARENT);
      }
      sh->anc[i] = m;
    }
  }
  // rows outside the Q box are zero so that their (unused) products stay finite
  for (int i = threadIdx.x; i < (128 - qrows) * 16; i += blockDim.x) {
    const int row = qrows + i / 16, c = i % 16;
    *reinterpret_cast<uint4*>(sQ + (c >> 3) * 16384 + row * 128 + (c & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;

  if (warp == 0) {
    // ------------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&tm_kc);
      prefetch_tmap(&tm_vc);
      mbar_arrive_expect_tx(&sh->q_full, 2 * qrows * 128);
      tma_load_3d(sQ, &tm_q, &sh->q_full, 0, kvh * G, base + node0);
      tma_load_3d(sQ + 16384, &tm_q, &sh->q_full, 64, kvh * G, base + node0);
      int issued = 0;
      // paged: the page entries of tile j + 1 are fetched while tile j's slot is awaited
      const int nbox = paged ? kDKeys / p.cache_box : 0;
      const int32_t* bt = paged ? p.block_table + (size_t)r * p.max_pages : nullptr;
      int32_t pg_cur[4], pg_nxt[4];
      auto fetch_pages = [&](int t, int32_t (&dst)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // only entries that cover a cached position are read
          const int pos = t * kDKeys + i * p.cache_box;
          dst[i] = (i < nbox && t < nt_cache && pos < L) ? __ldg(bt + (pos >> p.page_shift)) : -1;
        }
      };
      if (paged) fetch_pages(t0, pg_cur);
      for (int j = 0; j < T; ++j) {
        const int t = t0 + j;
        const int st = j % kDStages;
        const uint32_t ph = (j / kDStages) & 1;
        if (paged) fetch_pages(t + 1, pg_nxt);
        if (j >= kDStages && !mbar_wait(&sh->kv_empty[st], ph ^ 1)) {
          report(p.ws, ETREE_ETIMEOUT, DET_WAIT_ATTN);
          break;
        }
        uint8_t* dst = sKV + st * kDKV;
        uint64_t* full = &sh->kv_full[st];
        mbar_arrive_expect_tx(full, kDKV);
        if (t < nt_cache && !paged) {
          const int32_t slot = static_cast<int32_t>(sbase + (int64_t)t * kDKeys);
          tma_load_3d(dst, &tm_kc, full, 0, kvh, slot);
          tma_load_3d(dst + kDBox, &tm_kc, full, 64, kvh, slot);
          tma_load_3d(dst + 2 * kDBox, &tm_vc, full, 0, kvh, slot);
          tma_load_3d(dst + 3 * kDBox, &tm_vc, full, 64, kvh, slot);
        } else if (t < nt_cache) {
          // paged: 64 / cache_box boxes per half, each inside one page.  A page behind the last
          // cached key, or an entry outside the pool (reported), reads as zeros: its box lies
          // past the tensor.
          const int cb = p.cache_box, P = 1 << p.page_shift;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= nbox) break;
            const int pos = t * kDKeys + i * cb;
            int32_t page = pg_cur[i];
            if (page < 0 || (int64_t)page * P >= p.cache_slots) {
              if (pos < L) report(p.ws, ETREE_EDEVICE, DET_BAD_PAGE);
              page = (int32_t)(p.cache_slots >> p.page_shift);
            }
            const int32_t slot = page * P + (pos & (P - 1));
            const uint32_t off = (uint32_t)(i * cb * 128);
            tma_load_3d(dst + off, &tm_kc, full, 0, kvh, slot);
            tma_load_3d(dst + kDBox + off, &tm_kc, full, 64, kvh, slot);
            tma_load_3d(dst + 2 * kDBox + off, &tm_vc, full, 0, kvh, slot);
            tma_load_3d(dst + 3 * kDBox + off, &tm_vc, full, 64, kvh, slot);
          }
        } else {
          tma_load_3d(dst, &tm_kt, full, 0, kvh, base);
          tma_load_3d(dst + kDBox, &tm_kt, full, 64, kvh, base);
          tma_load_3d(dst + 2 * kDBox, &tm_vt, full, 0, kvh, base);
          tma_load_3d(dst + 3 * kDBox, &tm_vt, full, 64, kvh, base);
        }
        if (paged) {
#pragma unroll
          for (int i = 0; i < 4; ++i) pg_cur[i] = pg_nxt[i];
        }
        issued = j + 1;
      }
      // Before the CTA may exit, every copy into shared memory has landed: the last kDStages
      // loads (earlier ones were consumed, which implies landed) and Q.  Bounded, like all waits.
      bool drained = mbar_wait(&sh->q_full, 0);
      for (int j = issued > kDStages ? issued - kDStages : 0; j < issued; ++j)
        drained = mbar_wait(&sh->kv_full[j % kDStages], (j / kDStages) & 1) && drained;
      if (!drained) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_ATTN);
    }
  } else if (warp == 1 || warp == 2) {
    // --------------------------------------------------------------- MMA issuers, one per map
    // The warp stays converged and one elected lane issues (see elect_one).
    const int m = warp - 1;
    const uint32_t idS = idesc_bf16_f32(128, kDKeys);
    const uint32_t idO = idesc_bf16_f32(128, 128) | (1u << 16);     // B (V) is MN-major
    const uint64_t dq = smem_desc_sw128(sQ + m * 16384), dk0 = smem_desc_sw128(sKV + m * kDBox);
    const uint64_t dv0 = smem_desc_sw128_mn(sKV + 2 * kDBox, kDBox);
    bool ok = mbar_wait(&sh->q_full, 0);
    int ks = 0;                                         // the next K tile's stage and phase
    uint32_t kph = 0;
    auto qk = [&](int j) -> bool {
      if (!mbar_wait(&sh->kv_full[ks], kph)) return false;
      tc_fence_after();
      const uint64_t dk = dk0 + (uint64_t)(ks * (kDKV >> 4));
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_bf16(tmem + kDS + 128 * m + 64 * (j & 1), dq + 2 * k, dk + 2 * k, idS,
                      k > 0 ? 1u : 0u);
        tc_commit(&sh->s_full[m][j & 1]);
      }
      __syncwarp();
      if (++ks == kDStages) { ks = 0; kph ^= 1; }
      return true;
    };
    ok = ok && qk(0);
    if (T > 1) ok = ok && qk(1);
    int vs = 0;
    for (int j = 0; ok && j < T; ++j) {
      const int b = j & 1, t = t0 + j;
      const uint32_t ph = (j >> 1) & 1;
      // each map's warps clean one half of V in a tile with masked keys: both must be done.  These
      // tiles (at most the cache's last and the tree's) have a barrier each that completes once, since
      // the maps may run apart by more than the two tiles that p_full's phases tell from each other.
      const bool masked = t >= nt_cache || L - t * kDKeys < kDKeys;
      if (!mbar_wait(&sh->p_full[m][b], ph)) { ok = false; break; }
      if (masked && !mbar_wait(&sh->v_clean[t >= nt_cache], 0)) { ok = false; break; }
      tc_fence_after();
      const uint64_t dv = dv0 + (uint64_t)(vs * (kDKV >> 4));
      const uint32_t pa = tmem + kDS + 128 * m + 64 * b;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kDKeys / 16; ++k)
          tc_mma_bf16_ts(tmem + 128 * m, pa + 8 * k, dv + k * (2048 >> 4), idO,
                         (j > 0 || k > 0) ? 1u : 0u);
#pragma unroll
        for (int k = 0; k < kDKeys / 16; ++k)           // what the first part left
          tc_mma_bf16_ts(tmem + 128 * m, pa + 32 + 8 * k, dv + k * (2048 >> 4), idO, 1u);
        tc_commit(&sh->o_done[m]);
        if (j + 1 == T) tc_commit(&sh->o_final[m]);
        tc_commit(&sh->kv_empty[vs]);
      }
      __syncwarp();
      if (++vs == kDStages) vs = 0;
      // S of tile j + 2 takes the buffer that P of tile j was read from (and after the last tile
      // no MMA is in flight when TMEM is released)
      if (!mbar_wait(&sh->o_done[m], j & 1)) { ok = false; break; }
      if (j + 2 < T) ok = qk(j + 2);
    }
    if (!ok) {                                          // what was issued ends before TMEM goes
      if (elect_one()) tc_commit(&sh->drain[m]);
      __syncwarp();
      mbar_wait(&sh->drain[m], 0);
      if (lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_ATTN);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------- softmax warps
    const int m = (warp - 4) >> 2;                      // the map of this warp
    const int wq = warp & 3;                            // its TMEM lane quarter
    const int row = wq * 32 + lane;
    const int node_l = row / G, g = row - node_l * G;
    const int node = node0 + node_l;
    const bool valid = row < qrows && node < n;
    const bool work = __any_sync(0xffffffffu, valid);
    const uint64_t anc = (has_tree && valid) ? sh->anc[node] : 0ull;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    const float sl = p.scale_log2;
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < T; ++j) {
      const int t = t0 + j;
      const uint32_t buf = lane_base + kDS + 128 * m + 64 * (j & 1);
      if (!mbar_wait(&sh->s_full[m][j & 1], (j >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      float sc[64];
      if (work) tmem_ld64(buf, sc);

      const int lim = t < nt_cache ? min(kDKeys, L - t * kDKeys) : n;   // rows of the tile in use
      const bool masked = t >= nt_cache || lim < kDKeys;
      if (masked) {
        // this map's warps clean half m of the tile's V (see the header)
        if (!mbar_wait(&sh->kv_full[j % kDStages], (j / kDStages) & 1)) { ok = false; break; }
        uint8_t* v = sKV + (j % kDStages) * kDKV + (2 + m) * kDBox;
        unsigned long long bad = 0ull;
#pragma unroll 1
        for (int c = row; c < kDKeys * 8; c += 128) {   // 16-byte chunks, 8 a row
          uint4* at = reinterpret_cast<uint4*>(v + c * 16);
          const int key = c >> 3;
          if (key >= lim) {
            *at = make_uint4(0u, 0u, 0u, 0u);
          } else if (t >= nt_cache) {
            uint4 x = *at;
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            bool hit = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (bf16_nonfinite(w[i])) { w[i] &= 0xffff0000u; hit = true; }
              if (bf16_nonfinite(w[i] >> 16)) { w[i] &= 0x0000ffffu; hit = true; }
            }
            if (hit) {
              *at = make_uint4(w[0], w[1], w[2], w[3]);
              bad |= 1ull << key;
            }
          }
        }
        if (bad) atomicOr(&sh->bad, bad);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->v_clean[t >= nt_cache]);
      }
      if (work) {
        if (masked) {
          uint64_t kw;                                  // bit c: key c of the tile is visible
          if (t >= nt_cache) kw = anc;
          else kw = valid ? (1ull << lim) - 1ull : 0ull;            // 0 < lim < 64
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!((kw >> c) & 1ull)) sc[c] = -INFINITY;
        }
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          mx0 = fmax3(mx0, sc[c], sc[c + 1]);
          mx1 = fmax3(mx1, sc[c + 2], sc[c + 3]);
        }
        const float tms = fmaxf(mx0, mx1) * sl;         // row maximum in log2 units (sl > 0)
        const bool need = tms > m_ref + kDLazy;         // also true for the first finite maximum
        const bool any = __any_sync(0xffffffffu, need);
        const float m_new = need ? tms : m_ref;
        const float off = m_new == -INFINITY ? 0.f : m_new;
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {          // 32 keys: 16 columns of bf16 pairs
          uint32_t hi[16], lo[16];                      // P's first part, and what it leaves
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const float* z = sc + 32 * half + 2 * c;
            float x0, x1, x2, x3;
            ffma2(x0, x1, z[0], z[1], sl, -off);
            ffma2(x2, x3, z[2], z[3], sl, -off);
            const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
            const float e2 = ex2_approx(x2), e3 = ex2_approx(x3);
            fadd2(a0, a1, e0, e1);
            fadd2(a0, a1, e2, e3);
            hi[c] = upper_pair(e0, e1);
            hi[c + 1] = upper_pair(e2, e3);
            lo[c] = lower_pair(e0, e1);
            lo[c + 1] = lower_pair(e2, e3);
          }
          tmem_st16_async(buf + 16 * half, hi);
          tmem_st16_async(buf + 32 + 16 * half, lo);
        }
        const float corr = need ? ex2_approx(m_ref - m_new) : 1.f;
        l = l * corr + (a0 + a1);
        m_ref = m_new;
        // A rescale of O_m needs every earlier product of this map finished.  The one of tile j - 2
        // is: S of tile j was issued behind it.
        if (any && j >= 1) {
          if (!mbar_wait(&sh->o_done[m], (j - 1) & 1)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            const uint32_t ta = lane_base + 128 * m + c * 32;
            tmem_ld32(ta, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= corr;
            tmem_st32(ta, o);
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full[m][j & 1]);
    }
    // not o_done: its product of tile T - 2 may still run, and that phase would pass for T - 1's
    if (ok && !mbar_wait(&sh->o_final[m], 0)) ok = false;
    if (!ok) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_ATTN);
    tc_fence_after();
    const int h = kvh * G + g;
    const size_t gidx = (size_t)(base + (valid ? node : 0)) * p.hq + (valid ? h : 0);
    sh->l[m][row] = l;
    softmax_warps_sync();                               // both maps' O, sums and `bad` are final
    tc_fence_after();
    // columns [c0, c0 + 32) of O_mm, with the values taken out of the tree tile put back
    auto load_o = [&](int mm, int c0, float (&o)[32]) {
      __syncwarp();
      tmem_ld32(lane_base + 128 * mm + c0, o);
      unsigned long long fix = valid ? (sh->bad & anc) : 0ull;
      while (fix) {
        const int b = __ffsll((long long)fix) - 1;
        fix &= fix - 1ull;
        const uint16_t* vr = p.v_tree + (int64_t)(base + b) * p.v_stride + (int64_t)kvh * 128 + c0;
        for (int i = 0; i < 32; ++i)
          if (bf16_nonfinite(vr[i])) o[i] += bf16_bits(vr[i]);
      }
    };
    if (p.nsplit == 1) {
      // map m's warps finish dims [64 m, 64 m + 64)
      const float l0 = sh->l[0][row], l1 = sh->l[1][row];
      const float w0 = 1.f / l0, w1 = valid ? -p.lambda[h] / l1 : 0.f;
      float d[64], sq = 0.f;
      if (work) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float o0[32], o1[32];
          load_o(0, 64 * m + 32 * c, o0);
          load_o(1, 64 * m + 32 * c, o1);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float x = diff2(o0[i], w0, o1[i], w1);
            d[32 * c + i] = x;
            sq += x * x;
          }
        }
      }
      float mul = p.out_scale;
      if (p.norm_w) {
        sh->sq[m][row] = sq;
        softmax_warps_sync();
        mul *= rsqrtf((sh->sq[0][row] + sh->sq[1][row]) * (1.f / 128.f) + p.norm_eps);
      }
      if (valid) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + gidx * 128 + 64 * m);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float y[8];
          if (p.norm_w) {
            const uint4 wv = __ldg(reinterpret_cast<const uint4*>(p.norm_w + 64 * m) + q);
            const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[2 * i] = d[8 * q + 2 * i] * mul * bf16_bits(ww[i] & 0xffffu);
              y[2 * i + 1] = d[8 * q + 2 * i + 1] * mul * bf16_bits(ww[i] >> 16);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = d[8 * q + i] * mul;
          }
          dst[q] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                              pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        }
        if (p.lse) p.lse[gidx * 2 + m] = (m_ref + log2f(l)) * 0.69314718055994531f;
      }
    } else if (work) {
      float* op = p.o_part + ((gidx * p.nsplit + s) * 2 + m) * 128;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[32];
        load_o(m, 32 * c, o);
        if (valid) {
          float4* dst = reinterpret_cast<float4*>(op + 32 * c);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      if (valid) p.ml_part[(gidx * p.nsplit + s) * 2 + m] = make_float2(m_ref, l);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kDCols);
  }
}

// Merge of the split partials: one warp per (node, head), each lane 4 of the 128 dims.  Each map
// is merged by log-sum-exp in split order, then the difference, its norm and the one rounding.
constexpr int kDBatch = 4;                              // splits whose loads are in flight

__global__ void __launch_bounds__(256) attn_diff_combine_kernel(DiffParams p) {
  pdl_wait();
  pdl_trigger();
  const int gw = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (gw >= p.n_total * p.hq) return;
  const int node = gw / p.hq, h = gw - node * p.hq;
  int lo = 0, hi = p.B - 1;                             // request of this node
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_nodes[mid] <= node) lo = mid; else hi = mid - 1;
  }
  const int base = p.cu_nodes[lo], n = p.cu_nodes[lo + 1] - base;
  const int L = p.kv_len[lo];
  if (node < base || node >= base + n) return;          // behind the last request
  if (!diff_valid(p, base, n, L, p.block_table ? 0 : p.slot_base[lo])) return;   // reported above
  const int total = (L + kDKeys - 1) / kDKeys + 1;
  const int used = (total + p.tps - 1) / p.tps;         // the other splits hold stale values
  const float2* mlp = p.ml_part + (size_t)gw * p.nsplit * 2;
  const float4* op = reinterpret_cast<const float4*>(p.o_part + (size_t)gw * p.nsplit * 256);
  float M[2] = {-INFINITY, -INFINITY};
  for (int i = lane; i < used; i += 32) {
#pragma unroll
    for (int m = 0; m < 2; ++m) M[m] = fmaxf(M[m], mlp[2 * i + m].x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int m = 0; m < 2; ++m) M[m] = fmaxf(M[m], __shfl_xor_sync(0xffffffffu, M[m], off));
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  float ls[2] = {0.f, 0.f};
  const float Mb[2] = {M[0] == -INFINITY ? 0.f : M[0], M[1] == -INFINITY ? 0.f : M[1]};
  for (int s0 = 0; s0 < used; s0 += kDBatch) {
    float4 v[kDBatch][2];
    float2 ml[kDBatch][2];
#pragma unroll
    for (int i = 0; i < kDBatch; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (s0 + i < used) {
          v[i][m] = op[(size_t)(s0 + i) * 64 + m * 32 + lane];
          ml[i][m] = mlp[2 * (s0 + i) + m];
        }
#pragma unroll
    for (int i = 0; i < kDBatch; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (s0 + i < used) {
          const float w = exp2f(ml[i][m].x - Mb[m]);
          ls[m] += w * ml[i][m].y;
          acc[m].x += v[i][m].x * w;
          acc[m].y += v[i][m].y * w;
          acc[m].z += v[i][m].z * w;
          acc[m].w += v[i][m].w * w;
        }
  }
  const float w0 = 1.f / ls[0], w1 = -p.lambda[h] / ls[1];
  float d[4] = {diff2(acc[0].x, w0, acc[1].x, w1), diff2(acc[0].y, w0, acc[1].y, w1),
                diff2(acc[0].z, w0, acc[1].z, w1), diff2(acc[0].w, w0, acc[1].w, w1)};
  float mul = p.out_scale;
  if (p.norm_w) {
    float sq = d[0] * d[0] + d[1] * d[1] + d[2] * d[2] + d[3] * d[3];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, off);
    mul *= rsqrtf(sq * (1.f / 128.f) + p.norm_eps);
    const uint2 wv = __ldg(reinterpret_cast<const uint2*>(p.norm_w) + lane);
    d[0] *= bf16_bits(wv.x & 0xffffu);
    d[1] *= bf16_bits(wv.x >> 16);
    d[2] *= bf16_bits(wv.y & 0xffffu);
    d[3] *= bf16_bits(wv.y >> 16);
  }
  reinterpret_cast<uint2*>(p.out + (size_t)gw * 128)[lane] =
      make_uint2(pack_bf16x2(d[0] * mul, d[1] * mul), pack_bf16x2(d[2] * mul, d[3] * mul));
  if (p.lse && lane < 2)
    p.lse[(size_t)gw * 2 + lane] = lane == 0 ? (M[0] + log2f(ls[0])) * 0.69314718055994531f
                                             : (M[1] + log2f(ls[1])) * 0.69314718055994531f;
}

cudaError_t launch_attn_diff(const CUtensorMap& q, const CUtensorMap& kc, const CUtensorMap& vc,
                             const CUtensorMap& kt, const CUtensorMap& vt, const DiffParams& p,
                             cudaStream_t stream) {
  const size_t smem = 1024 + kDQ + (size_t)kDStages * kDKV + sizeof(DiffSmem);
  cudaError_t e = raise_smem_once(attn_diff_kernel, (int)smem);
  if (e != cudaSuccess) return e;
  dim3 grid(p.B * p.hkv * p.mchunks, p.nsplit);
  attn_diff_kernel<<<grid, kDThreads, smem, stream>>>(q, kc, vc, kt, vt, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.nsplit == 1) return e;
  const int64_t blocks = ((int64_t)p.n_total * p.hq * 32 + 255) / 256;
  return launch_pdl(attn_diff_combine_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, p);
}

}  // namespace etree
