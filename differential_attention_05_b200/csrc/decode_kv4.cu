// decode_kv4.cu -- split-KV differential attention decode over a cache held in 4 bits (the
// record: kv4.cuh), V1 and V2, contiguous and paged.
//
// With s the scales and n the nibbles of the records, q one query row of a KV head,
//   x_t = c sum_g sK[t,g] sum_{i in g} q_i (nK[t,i] - 8),       c = log2(e) / sqrt(d)
//   O   = sum_t 2^(x_t - M) sV[t,g] (nV[t,:] - 8) / sum_t 2^(x_t - M),
// and out = O_1 - lambda O_2 for the two branches ("Differential Attention (V2)", The
// Concept). V1 is the same with two rows for each head: branch 1 is (q_1 | 0) and branch 2
// (0 | q_2) over the cached row (K_1 | K_2), and the norm and scale follow.
//
// One block takes (batch entry, KV head, split of the keys, up to 8 NT query rows). Its four
// warps work alone, each on 32 keys of every 128: a ring of cp.async stages of its own, its
// own running maximum, sums and output; the block joins them at the end, a second kernel
// joins the splits. Products run on mma.sync m16n8k16 in fp16 with fp32 sums, keys (or value
// channels) as the 16 rows and query rows as the 8 columns:
//   * Codes go from shared memory to registers by ldmatrix (keys: one 16-byte group of a row
//     per matrix row, a thread gets 8 channels of one key; values: transposed, a thread gets
//     4 channels of two neighbouring keys, which is the pair an MMA operand register holds).
//   * K nibbles are used as fp16 subnormals: n in the low mantissa bits is n 2^-24, the next
//     nibble 16 n 2^-24 against q / 16, so unpacking is one AND for two channels. The -8 is
//     the accumulators' start, -8 * 2^-24 sum q: exact up to the fp32 sums, since half the
//     range is all that cancels.
//   * V nibbles become n - 8 exactly (0x6400 | n is 1024 + n). Left as subnormals with the -8
//     from a second MMA over constants the full step took 455 us instead of 469, but the
//     cancelling sums lost up to 2^-16 of a scale, which shows where a peaked row's key has
//     the code 0.
//   * Scales stay outside the MMAs: a group is two k-steps, its fp32 sums are scaled and
//     added; for V the probability is multiplied by the scale in fp32 and rounded to fp16
//     once (2^-12 relative; bf16's 2^-9 would be amplified by the subtraction and V1's norm).
//     fp16's range is kept by the running maximum: M bounds x + E, E the exponent of the
//     chunk's largest V scale, so products lie under 2^(kTop + kSlack) = 2^15, and M is
//     raised only when the bound would be passed. Products under 2^-22 of the largest
//     probability times the largest scale become subnormal and lose bits.
//   * q is taken times a power of two per row so that its largest element is in [2^14, 2^15);
//     fp16 then holds every element above 2^-31 of the largest exactly.
#include <cuda_fp16.h>

#include <string.h>

#include "kv4.cuh"
#include "tma_host.cuh"

namespace diffattn {

namespace {
constexpr int W = kKv4Width;
constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int KEYS = 32;                            // keys of a warp's chunk
constexpr int STAGES = 4;
constexpr int STAGE_BYTES = KEYS * kKv4Record;      // 4608
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int SMEM_BYTES = WARPS * RING_BYTES;      // 73728
constexpr float kTop = 8.f;                         // p * scale <= 2^kTop when M is raised ...
constexpr float kSlack = 7.f;                       // ... and <= 2^(kTop + kSlack) before
static_assert(kKv4Chunk == WARPS * KEYS, "a block's keys");
static_assert(W == THREADS, "one thread per value channel in the joins");
static_assert(STAGE_BYTES % 128 == 0 && (8 * kKv4Record) % 128 == 0, "TMA destinations");

// How a chunk reaches shared memory: TMA boxes of 32 records (contiguous) or of a page's run
// of up to 32 (pages of 8 tokens and more; a box of fewer would not end on a 128-byte
// boundary), or 16-byte copies (smaller pages, and strides that TMA does not take).
enum Kv4Load { kTma, kTmaPaged, kCopy };
}  // namespace

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// d = a b + c
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// the even and the odd nibbles of the low byte of each half of w, as fp16: n 2^-24, 16 n 2^-24
__device__ __forceinline__ uint32_t nib_even(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t nib_odd(uint32_t w) { return w & 0x00f000f0u; }
// transpose of an 8 x 8 matrix of 16-bit elements held one row per four lanes
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// the same nibbles minus 8, exact: 1024 + n - 1032 and (1024 + 16 n) / 16 - 72
__device__ __forceinline__ uint32_t code_even(uint32_t w) {
  const uint32_t x = (w & 0x000f000fu) | 0x64006400u;
  const __half2 y = __hadd2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(-1032.f));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t code_odd(uint32_t w) {
  const uint32_t x = (w & 0x00f000f0u) | 0x64006400u;
  const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(0.0625f),
                            __float2half2_rn(-72.f));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The output of one unit (V1 head or V2 pair) from its branches' attention outputs, channel
// `c` of the W threads with `mine`: the difference, and V1's norm and scale. All threads of the
// block take part; `red` holds 4 floats.
__device__ __forceinline__ void store_unit(const DecodeKv4Args& a, int b, int u, int c, bool mine, float o1,
                                           float o2, float* red) {
  float y = o1 - __ldg(a.lambda + u) * o2;
  if (a.apply_norm) {
    const float ss = warp_sum(y * y);
    if (mine && (c & 31) == 0) red[c >> 5] = ss;
    __syncthreads();
    const float tot = (red[0] + red[1]) + (red[2] + red[3]);
    __syncthreads();
    y = y * rsqrtf(tot * (1.f / W) + a.eps) * (1.f - __ldg(a.lambda_init));
  }
  const int64_t off = b * a.os[0] + (int64_t)u * a.os[1] + c;
  if (mine && in_bounds(off, 1, a.ext_out, a.cache.dev_status, a.cache.dbg_status))
    static_cast<__nv_bfloat16*>(a.out)[off] = __float2bfloat16_rn(y);
}

// missing[s] = v and missing[s] with the array in registers
template <int N>
__device__ __forceinline__ void set_stage(uint32_t (&m)[N], int s, uint32_t v) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i == s) m[i] = v;
}
template <int N>
__device__ __forceinline__ uint32_t get_stage(const uint32_t (&m)[N], int s) {
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i == s) v = m[i];
  return v;
}

template <int NT, Kv4Load LOAD>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 3 : 2)
    decode_kv4_split_kernel(const __grid_constant__ CUtensorMap map, DecodeKv4Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t landed[WARPS][STAGES];  // TMA: the chunk in a stage has arrived
  __shared__ int abort_flag;
  __shared__ float red[4];
  const int tiles = (a.group + 8 * NT - 1) / (8 * NT);
  const int g = blockIdx.x / tiles, row0 = (blockIdx.x % tiles) * 8 * NT;  // KV head, first query row
  const int split = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;  // fragment row (or column) and pair index

  // device-side lengths are clamped into [0, L] so a bad value cannot read past the cache
  const int kv_len = a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.cache.L) : a.cache.L;
  const int t_begin = split * a.split_len;
  const int t_end = min(t_begin + a.split_len, kv_len);
  const int w_begin = t_begin + warp * KEYS;
  const int n_chunks = t_end > w_begin ? (t_end - w_begin + kKv4Chunk - 1) / kKv4Chunk : 0;  // of this warp

  uint8_t* ring = smem + warp * RING_BYTES;
  [[maybe_unused]] const int64_t head_off = (int64_t)g * a.cache.stride[2];
  bool bad_page = false;

  // Paged: the pages of a chunk are looked up one chunk ahead of its copies. kTmaPaged: lane i
  // holds box i's page; kCopy: lane r the byte offset of record r. -1: no key there, -2:
  // a page outside the pool. Either way the records' scales become zero, so they count as K
  // and V rows of zeros (and keys past the end get no weight at all).
  const int box_rows = LOAD == kTmaPaged ? min(1 << a.cache.page_shift, KEYS) : KEYS;
  int64_t ahead = -1;
  auto lookup = [&](int c) {
    const int tok0 = w_begin + c * kKv4Chunk;
    ahead = -1;
    if constexpr (LOAD == kTmaPaged) {
      const int tok = tok0 + lane * box_rows;
      if (lane * box_rows < KEYS && tok < t_end) {
        const int64_t bi = (int64_t)b * a.cache.bt_stride + (tok >> a.cache.page_shift);
        int id = -1;
        if (in_bounds(bi, 1, a.cache.ext_bt, a.cache.dev_status, a.cache.dbg_status))
          id = __ldg(a.cache.block_table + bi);
        ahead = (unsigned)id < (unsigned)a.cache.num_pages ? id : -2;
      }
    } else if constexpr (LOAD == kCopy) {
      if (tok0 + lane < t_end) {
        ahead = kv4_page_offset(a.cache, b, tok0 + lane);
        if (ahead < 0) ahead = -2;
      }
    }
    bad_page = bad_page || ahead == -2;
  };
  // bit s * KEYS.. : rows of the chunk in stage s that a bad page left out
  uint32_t missing[LOAD == kTma ? 1 : STAGES];
  auto load = [&](int c) {
    const int s = c % STAGES;
    uint8_t* st = ring + s * STAGE_BYTES;
    const int tok0 = w_begin + c * kKv4Chunk;
    if constexpr (LOAD == kTma) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&landed[warp][s], STAGE_BYTES);
        tma_load_4d(st, &map, &landed[warp][s], 0, g, tok0, b);
      }
    } else if constexpr (LOAD == kTmaPaged) {
      const uint32_t boxes = __ballot_sync(0xffffffffu, ahead >= 0);
      uint32_t bad = __ballot_sync(0xffffffffu, ahead == -2);
      if (lane == 0) mbar_arrive_expect_tx(&landed[warp][s], __popc(boxes) * box_rows * kKv4Record);
      __syncwarp();
      if (ahead >= 0)
        tma_load_4d(st + lane * box_rows * kKv4Record, &map, &landed[warp][s], 0, g,
                    (tok0 + lane * box_rows) & ((1 << a.cache.page_shift) - 1), (int)ahead);
      uint32_t rows = 0;
      while (bad) {  // a bad box's rows
        const int i = __ffs(bad) - 1;
        bad &= bad - 1;
        rows |= (box_rows == 32 ? 0xffffffffu : (1u << box_rows) - 1u) << (i * box_rows);
      }
      set_stage(missing, s, rows);
    } else {
      // eight lanes take the 128 code bytes of a record, four records at a time, then lane r
      // the scales of record r
      auto copy = [&](int row, int64_t row_off, int part) {
        bool ok = row_off >= 0;
        const int64_t off = (ok ? row_off : 0) + head_off + part * 16;
        ok = ok && in_bounds(off, 16, a.cache.ext, a.cache.dev_status, a.cache.dbg_status);
        cp_async_16(st + row * kKv4Record + part * 16, a.cache.base + (ok ? off : 0), ok ? 16u : 0u);
      };
#pragma unroll
      for (int it = 0; it < KEYS / 4; ++it) {
        const int row = it * 4 + (lane >> 3);
        copy(row, __shfl_sync(0xffffffffu, ahead, row), lane & 7);
      }
      copy(lane, ahead, 8);
    }
  };

  if (a.splits > 1) cudaTriggerProgrammaticLaunchCompletion();
  if constexpr (LOAD != kCopy) {
    if (lane < STAGES) mbar_init(&landed[warp][lane], 1);
    if (tid == 0) abort_flag = 0;
    fence_barrier_init();
    __syncthreads();
  }
  lookup(0);
#pragma unroll
  for (int c = 0; c < STAGES - 1; ++c) {
    if (c < n_chunks) {
      load(c);
      lookup(c + 1);
    }
    if constexpr (LOAD == kCopy) cp_async_commit();
  }

  // Query fragments (B operands), rows scaled to fp16: for group gr and k-step ks, register 0
  // holds channels 32 gr + 8 tq + 2 ks + {0, 4}, register 1 the next pair over 16 (the order
  // in which the nibbles of a word come). Lane column gq; start and factor are per column of
  // the accumulators, 2 tq and 2 tq + 1.
  uint32_t qb[NT][8][2];
  float start[NT][4][4];  // -8 * 2^-24 * sum of the group's q, as accumulators
  float factor[NT][2];    // accumulated score -> log2 domain
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = row0 + nt * 8 + gq;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    int64_t off = b * a.qs[0];
    if (a.v1) off += (int64_t)g * a.qs[1];  // the branches lie side by side in the head's row
    else off += ((int64_t)g * a.group + row) * a.qs[1];
    const bool ok = row < a.group && in_bounds(off, W, a.ext_q, a.cache.dev_status, a.cache.dbg_status);
    uint4 w[4];
    float top = 0.f;
    bool odd = false;  // an infinity or a NaN
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      // V1: row 0 has only groups 0, 1 (branch 1), row 1 only groups 2, 3 (branch 2)
      const bool mine = ok && (!a.v1 || (gr >> 1) == row);
      w[gr] = mine ? *reinterpret_cast<const uint4*>(q + off + gr * 32 + tq * 8) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t x[4] = {w[gr].x, w[gr].y, w[gr].z, w[gr].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top = fmaxf(top, fmaxf(fabsf(bf16_low(x[i])), fabsf(bf16_high(x[i]))));
        odd = odd || (x[i] & 0x7f80u) == 0x7f80u || (x[i] & 0x7f800000u) == 0x7f800000u;
      }
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // exponent field of the row's largest element -> scale 2^(141 - ex), inverse in `factor`
    const int ex = (int)(__float_as_uint(top) >> 23);
    const float up = odd ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)min(268 - ex, 254) << 23);
    float sums[4];
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      const uint32_t x[4] = {w[gr].x, w[gr].y, w[gr].z, w[gr].w};
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_low(x[i]) * up;
        v[2 * i + 1] = bf16_high(x[i]) * up;
      }
      float sum = 0.f;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        qb[nt][2 * gr + ks][0] = pack_f16(v[2 * ks], v[2 * ks + 4]);
        qb[nt][2 * gr + ks][1] = pack_f16(v[2 * ks + 1] * 0.0625f, v[2 * ks + 5] * 0.0625f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sums[gr] = sum * (-8.f / 16777216.f);
    }
    // 2^24 (nibbles as 2^-24) * 2^(ex - 141) * log2(e) / sqrt(d). Rows with elements past
    // 2^117 overflow here to infinite scores
    const float down = ldexpf(1.4426950408889634f * (a.v1 ? 0.125f : 0.08838834764831845f),
                              24 - 141 + max(ex, 14));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int from = (2 * tq + j) * 4;  // a lane of column 2 tq + j
      factor[nt][j] = __shfl_sync(0xffffffffu, down, from);
#pragma unroll
      for (int gr = 0; gr < 4; ++gr)
        start[nt][gr][j] = start[nt][gr][2 + j] = __shfl_sync(0xffffffffu, sums[gr], from);
    }
  }

  float m[NT][2], bias[NT][2], l[NT][2];  // columns 2 tq, 2 tq + 1: M, kTop - M, sum of p
  // [group][tile]: channels 32 g + 4 gq + 2 tile + {0, 1}
  float o[NT][4][2][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m[nt][j] = -INFINITY;
      bias[nt][j] = kTop;
      l[nt][j] = 0.f;
    }
#pragma unroll
    for (int gr = 0; gr < 4; ++gr)
#pragma unroll
      for (int ti = 0; ti < 2; ++ti)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][gr][ti][i] = 0.f;
  }

  for (int c = 0; c < n_chunks; ++c) {
    if (c + STAGES - 1 < n_chunks) {
      load(c + STAGES - 1);
      lookup(c + STAGES);
    }
    const int stage = c % STAGES;
    uint8_t* st = ring + stage * STAGE_BYTES;
    const int left = t_end - (w_begin + c * kKv4Chunk);  // keys of the chunk that exist
    if constexpr (LOAD == kCopy) {
      cp_async_commit();
      cp_async_wait<STAGES - 1>();
      __syncwarp();
    } else {
      const bool ok = mbar_wait(&landed[warp][stage], (c / STAGES) & 1, &abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        // a copy that never landed: let the ones in flight finish before the ring is reused
        const int issued = min(c + STAGES, n_chunks);
        for (int cc = c; cc < issued; ++cc) mbar_wait_drain(&landed[warp][cc % STAGES], (cc / STAGES) & 1);
        if (lane == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_TIMEOUT);
        break;
      }
      uint32_t out = 0;
      if constexpr (LOAD == kTmaPaged) out = get_stage(missing, stage);
      if (left < KEYS || out) {  // scales of records that are not there
        if (lane >= left || ((out >> lane) & 1u))
          *reinterpret_cast<uint4*>(st + lane * kKv4Record + kKv4Scales) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();  // before a later TMA copy rewrites the stage
        __syncwarp();
      }
    }
    const uint32_t st32 = smem_u32(st);

    // exponent bound of the chunk's V scales: |scale| < 2^E for all of them (bf16 bits are
    // ordered as magnitudes; not below -90, so that rows of zeros do not overflow p)
    const uint2 vs = *reinterpret_cast<const uint2*>(st + lane * kKv4Record + kKv4Scales + 8);
    uint32_t big = __vmaxu2(vs.x & 0x7fff7fffu, vs.y & 0x7fff7fffu);
    big = max(big & 0xffffu, big >> 16);
    big = __reduce_max_sync(0xffffffffu, big);
    const float E = fmaxf((float)((int)(big >> 7) - 126), -90.f);

    // scores of 2 x 16 keys: x[.][mt][0, 1] key mt * 16 + gq, [2, 3] key + 8, columns 2tq, +1
    float x[NT][2][4];
    uint4 scales[2][2];  // of those keys: {K 0 1, K 2 3, V 0 1, V 2 3}
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        scales[mt][h] =
            *reinterpret_cast<const uint4*>(st + (mt * 16 + h * 8 + gq) * kKv4Record + kKv4Scales);
      const uint32_t row = st32 + (mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * kKv4Record + (lane >> 4) * 16;
#pragma unroll
      for (int gp = 0; gp < 2; ++gp) {
        uint32_t r[4];
        ldsm4(row + gp * 32, r);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const int gr = 2 * gp + gg;
          const uint32_t lo = r[2 * gg], hi = r[2 * gg + 1], lo8 = lo >> 8, hi8 = hi >> 8;
          const uint32_t k0 = gp ? scales[mt][0].y : scales[mt][0].x, k1 = gp ? scales[mt][1].y : scales[mt][1].x;
          const float s0 = gg ? bf16_high(k0) : bf16_low(k0), s1 = gg ? bf16_high(k1) : bf16_low(k1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4];
            mma_f16(acc, nib_even(lo), nib_even(hi), nib_odd(lo), nib_odd(hi), qb[nt][2 * gr][0], qb[nt][2 * gr][1],
                    start[nt][gr]);
            mma_f16(acc, nib_even(lo8), nib_even(hi8), nib_odd(lo8), nib_odd(hi8), qb[nt][2 * gr + 1][0],
                    qb[nt][2 * gr + 1][1], acc);
            float* xx = x[nt][mt];
            if (gr == 0) {
              xx[0] = s0 * acc[0]; xx[1] = s0 * acc[1]; xx[2] = s1 * acc[2]; xx[3] = s1 * acc[3];
            } else {
              xx[0] = fmaf(s0, acc[0], xx[0]); xx[1] = fmaf(s0, acc[1], xx[1]);
              xx[2] = fmaf(s1, acc[2], xx[2]); xx[3] = fmaf(s1, acc[3], xx[3]);
            }
          }
        }
      }
    }

    // keys past the end get -inf; does any score pass its row's bound?
    bool raise = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (left < KEYS) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (mt * 16 + (i >> 1) * 8 + gq >= left) x[nt][mt][i] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float t = fmaxf(fmax3(x[nt][0][j], x[nt][0][2 + j], x[nt][1][j]), x[nt][1][2 + j]);
        top[nt][j] = fmaf(t, factor[nt][j], E);
        raise = raise || top[nt][j] > m[nt][j] + kSlack;
      }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float t = top[nt][j];
#pragma unroll
          for (int s = 4; s <= 16; s <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
          const float mn = fmaxf(m[nt][j], t);
          const float alpha = m[nt][j] == -INFINITY ? 0.f : ex2(m[nt][j] - mn);
          m[nt][j] = mn;
          bias[nt][j] = mn == -INFINITY ? kTop : kTop - mn;
          l[nt][j] *= alpha;
#pragma unroll
          for (int gr = 0; gr < 4; ++gr)
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {
              o[nt][gr][ti][j] *= alpha;
              o[nt][gr][ti][2 + j] *= alpha;
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[nt][mt][i] = ex2(fmaf(x[nt][mt][i], factor[nt][i & 1], bias[nt][i & 1]));
          l[nt][i & 1] += x[nt][mt][i];
        }

    // O += (p scale)^T-fragments times V
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t row = st32 + (mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * kKv4Record + kKv4VCodes + (lane >> 4) * 16;
#pragma unroll
      for (int gp = 0; gp < 2; ++gp) {
        uint32_t r[4];
        ldsm4_t(row + gp * 32, r);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const int gr = 2 * gp + gg;
          const uint32_t v0 = gp ? scales[mt][0].w : scales[mt][0].z, v1 = gp ? scales[mt][1].w : scales[mt][1].z;
          const float s0 = gg ? bf16_high(v0) : bf16_low(v0), s1 = gg ? bf16_high(v1) : bf16_low(v1);
          const uint32_t lo = r[2 * gg], hi = r[2 * gg + 1], lo8 = lo >> 8, hi8 = hi >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float* p = x[nt][mt];
            const uint32_t b0 = transpose8(pack_f16(p[0] * s0, p[1] * s0));
            const uint32_t b1 = transpose8(pack_f16(p[2] * s1, p[3] * s1));
            float(&o0)[4] = o[nt][gr][0];
            float(&o1)[4] = o[nt][gr][1];
            mma_f16(o0, code_even(lo), code_odd(lo), code_even(hi), code_odd(hi), b0, b1, o0);
            mma_f16(o1, code_even(lo8), code_odd(lo8), code_even(hi8), code_odd(hi8), b0, b1, o1);
          }
        }
      }
    }
    __syncwarp();  // the stage is refilled by the next iteration's copies
  }
  if constexpr (LOAD == kCopy) cp_async_wait<0>();
  if (bad_page) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);

  // join the warps: [warp][row][channel] outputs and their (M, l) in the ring's memory
  constexpr int ROWS = 8 * NT;
  float* sm_o = reinterpret_cast<float*>(smem);
  float* sm_ml = sm_o + WARPS * ROWS * W;
  static_assert(WARPS * ROWS * (W + 2) * 4 <= SMEM_BYTES, "the join fits in the ring");
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = warp * ROWS + nt * 8 + 2 * tq + j;
#pragma unroll
      for (int s = 4; s <= 16; s <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], s);
      if (gq == 0) {
        sm_ml[2 * row] = m[nt][j];
        sm_ml[2 * row + 1] = l[nt][j];
      }
#pragma unroll
      for (int gr = 0; gr < 4; ++gr)
        *reinterpret_cast<float4*>(sm_o + row * W + gr * 32 + gq * 4) =
            make_float4(o[nt][gr][0][j], o[nt][gr][0][2 + j], o[nt][gr][1][j], o[nt][gr][1][2 + j]);

    }
  __syncthreads();
  const int rows = min(ROWS, a.group - row0);
  float prev = 0.f;
  for (int r = 0; r < rows; ++r) {
    float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm_ml[2 * (w * ROWS + r)]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float mw = sm_ml[2 * (w * ROWS + r)];
      // a warp without keys, or with none above -inf, has M = -inf and nothing to add; only
      // a NaN among its sums is passed on
      const float f = mw == -INFINITY ? 1.f : ex2(mw - M);
      L = fmaf(sm_ml[2 * (w * ROWS + r) + 1], f, L);
      O = fmaf(sm_o[(w * ROWS + r) * W + tid], f, O);
    }
    if (a.splits == 1) {
      const float y = L == 0.f ? 0.f : O / L;
      if (r & 1) store_unit(a, b, a.v1 ? g : (g * a.group + row0 + r) >> 1, tid, true, prev, y, red);
      prev = y;
    } else {
      const int64_t rec = ((int64_t)b * a.H * a.group + g * a.group + row0 + r) * a.splits + split;
      if (in_bounds(rec * W + tid, 1, a.ext_ws_o, a.cache.dev_status, a.cache.dbg_status))
        a.ws_o[rec * W + tid] = O;
      if (tid == 0 && in_bounds(rec * 2, 2, a.ext_ws_ml, a.cache.dev_status, a.cache.dbg_status)) {
        a.ws_ml[rec * 2] = M;
        a.ws_ml[rec * 2 + 1] = L;
      }
    }
  }
}

// Joins the splits: one block per unit (V1 head or V2 pair) and batch entry. A split's weight
// 2^(M_s - M) is computed once by one thread; SLICES threads per value channel then add every
// SLICES-th split, both rows, and their sums are added in order. (With one thread per channel
// walking all splits the join of 103 splits took 52 us, more than the attention.)
constexpr int SLICES = 4;
constexpr int JOIN = 128;  // splits whose weights are held at a time
__global__ void __launch_bounds__(W * SLICES) decode_kv4_combine_kernel(DecodeKv4Args a) {
  __shared__ float weight[2][JOIN];
  __shared__ float part[SLICES][2][W];
  __shared__ float red[2][W * SLICES / 32];
  const int u = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, c = tid % W, slice = tid / W;
  const int64_t rec0 = ((int64_t)b * a.H * a.group + 2 * u) * a.splits;  // row 2u; row 2u + 1 follows
  cudaGridDependencySynchronize();  // the split kernel's states
  const bool ok =
      in_bounds(rec0 * 2, 4 * (int64_t)a.splits, a.ext_ws_ml, a.cache.dev_status, a.cache.dbg_status) &&
      in_bounds(rec0 * W, 2 * (int64_t)a.splits * W, a.ext_ws_o, a.cache.dev_status, a.cache.dbg_status);
  const int splits = ok ? a.splits : 0;
  const float* ml = a.ws_ml + rec0 * 2;
  const float* po = a.ws_o + rec0 * W + c;

  float M[2] = {-INFINITY, -INFINITY};
  for (int s = tid; s < splits; s += W * SLICES)
#pragma unroll
    for (int e = 0; e < 2; ++e) M[e] = fmaxf(M[e], ml[2 * (e * splits + s)]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    M[e] = warp_max(M[e]);
    if ((tid & 31) == 0) red[e][tid >> 5] = M[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int w = 0; w < W * SLICES / 32; ++w) M[e] = fmaxf(M[e], red[e][w]);

  float L = 0.f, O[2] = {0.f, 0.f};  // threads 0 .. 2 JOIN - 1: row tid / JOIN's sums
  for (int s0 = 0; s0 < splits; s0 += JOIN) {
    const int n = min(JOIN, splits - s0);
    __syncthreads();
    if (tid < 2 * JOIN && tid % JOIN < n) {
      const int e = tid / JOIN, s = tid % JOIN;
      const float2 v = *reinterpret_cast<const float2*>(ml + 2 * (e * splits + s0 + s));
      // a split without keys has M = -inf and nothing to add; only a NaN is passed on
      const float f = v.x == -INFINITY ? 1.f : ex2(v.x - (e ? M[1] : M[0]));
      weight[e][s] = f;
      L = fmaf(v.y, f, L);
    }
    __syncthreads();
#pragma unroll 4
    for (int s = slice; s < n; s += SLICES) {
      O[0] = fmaf(po[(int64_t)(s0 + s) * W], weight[0][s], O[0]);
      O[1] = fmaf(po[(int64_t)(splits + s0 + s) * W], weight[1][s], O[1]);
    }
  }
  L = warp_sum(L);
  __syncthreads();
  if ((tid & 31) == 0) red[0][tid >> 5] = L;
  part[slice][0][c] = O[0];
  part[slice][1][c] = O[1];
  __syncthreads();
  float res[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < JOIN / 32; ++w) l += red[0][e * (JOIN / 32) + w];
#pragma unroll
    for (int i = 0; i < SLICES; ++i) o += part[i][e][c];
    res[e] = l == 0.f ? 0.f : o / l;
  }
  store_unit(a, b, u, c, slice == 0, res[0], res[1], red[1]);
}

// Splits of the keys: the count whose waves over the GPU's block slots take the least time, a
// block costing its keys and kSetup more for its start and join.
int decode_kv4_default_splits(int B, int L, int H, int group) {
  const int nt = group > 8 ? 2 : 1;
  const int64_t units = (int64_t)B * H * ((group + 8 * nt - 1) / (8 * nt));
  const int64_t slots = 148 * (nt == 1 ? 3 : 2);
  const int64_t chunks = (L + kKv4Chunk - 1) / kKv4Chunk;
  const int64_t most = chunks < 256 ? chunks : 256;
  constexpr int64_t kSetup = 3;  // chunks
  int64_t best = 1, best_cost = -1;
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t waves = (units * s + slots - 1) / slots;
    const int64_t cost = waves * ((chunks + s - 1) / s + kSetup) + (s > 1 ? 2 : 0);
    if (best_cost < 0 || cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return (int)best;
}

// {144 bytes, heads, rows, entries or pages}, boxes of one head's `box` records; false where
// the strides are out of TMA's range
static bool kv4_map(CUtensorMap* m, const Kv4Cache& c, int H, int rows, int outer, int box) {
  auto fn = encode_fn();
  if (!fn || rows < 1) return false;
  int64_t hs = c.stride[2], ts = c.stride[1], os = c.stride[0];
  // extents of 1 may carry any stride; give TMA a well-formed one
  if (H == 1) hs = kKv4Record;
  if (rows == 1) ts = hs * H;
  if (outer == 1) os = ts * rows;
  const cuuint64_t dims[4] = {(cuuint64_t)kKv4Record, (cuuint64_t)H, (cuuint64_t)rows, (cuuint64_t)outer};
  const cuuint64_t strides[3] = {(cuuint64_t)hs, (cuuint64_t)ts, (cuuint64_t)os};
  const cuuint32_t boxes[4] = {(cuuint32_t)kKv4Record, 1, (cuuint32_t)box, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.base, dims, strides, boxes, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
static cudaError_t launch_split(const DecodeKv4Args& a, cudaStream_t stream) {
  const bool paged = a.cache.block_table != nullptr;
  const int page = 1 << a.cache.page_shift;
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  void (*fn)(CUtensorMap, DecodeKv4Args) = decode_kv4_split_kernel<NT, kCopy>;
  if (!paged && kv4_map(&map, a.cache, a.H, a.cache.L, a.B, KEYS)) {
    fn = decode_kv4_split_kernel<NT, kTma>;
  } else if (paged && page >= 8 && kv4_map(&map, a.cache, a.H, page, a.cache.num_pages, page < KEYS ? page : KEYS)) {
    fn = decode_kv4_split_kernel<NT, kTmaPaged>;
  }
  cudaError_t e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int tiles = (a.group + 8 * NT - 1) / (8 * NT);
  fn<<<dim3(a.H * tiles, a.splits, a.B), THREADS, SMEM_BYTES, stream>>>(map, a);
  return cudaGetLastError();
}

cudaError_t launch_decode_kv4(const DecodeKv4Args& a, cudaStream_t stream) {
  const cudaError_t e = a.group > 8 ? launch_split<2>(a, stream) : launch_split<1>(a, stream);
  if (e != cudaSuccess || a.splits == 1) return e;
  // launched while the last splits still run; the kernel waits for them itself
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(a.H * a.group / 2, a.B);
  cfg.blockDim = dim3(W * SLICES);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_kv4_combine_kernel, a);
}

}  // namespace diffattn
