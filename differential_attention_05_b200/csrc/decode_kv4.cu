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
constexpr int KEYS = 32;      // keys that a warp takes of a chunk
constexpr float kTop = 8.f;   // p * scale <= 2^kTop when M is raised ...
constexpr float kSlack = 7.f; // ... and <= 2^(kTop + kSlack) before
static_assert(W == THREADS, "one thread per value channel in the joins");

// A block takes HB neighbouring KV heads, WARPS / HB warps for each. A chunk is CK tokens in
// a stage of one row per token: the HB records side by side, as they lie in the cache, and 16
// bytes more (of the next record, unused) where that is needed for a pitch that is an odd
// number of 16-byte units, so that ldmatrix's 8 rows meet no bank twice.
template <int HB>
struct Tile {
  static constexpr int PER_HEAD = WARPS / HB;  // warps of a head
  static constexpr int CK = KEYS * PER_HEAD;
  static constexpr int PITCH = HB * kKv4Record + (HB == 1 ? 0 : 16);
  static constexpr int STAGES = HB == 2 ? 3 : 4;  // what shared memory holds for three blocks
  static constexpr int STAGE_BYTES = CK * PITCH;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES;
  static_assert((PITCH / 16) % 2 == 1 && STAGE_BYTES % 128 == 0 && 8 * PITCH % 128 == 0, "layout");
};

// How a chunk reaches shared memory: TMA boxes of CK rows (contiguous) or of a page's run of
// up to CK (pages of 8 tokens and more; a box of fewer would not end on a 128-byte boundary),
// or 16-byte copies (smaller pages, and strides that TMA does not take).
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
// (w & mask) | magic in one LOP3: the constants come in registers (`Magic`), because with two
// immediates the compiler makes two instructions of it, 64 more for a chunk's V codes
struct Magic {
  uint32_t even, odd, magic;
  __device__ Magic() {
    asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(even));
    asm volatile("mov.b32 %0, 0x00f000f0;" : "=r"(odd));
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
  }
};
__device__ __forceinline__ __half2 and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "r"(mask), "r"(magic));
  return *reinterpret_cast<const __half2*>(&x);
}
// the same nibbles minus 8, exact: 1024 + n - 1032 and (1024 + 16 n) / 16 - 72
__device__ __forceinline__ uint32_t code_even(uint32_t w, const Magic& k) {
  const __half2 y = __hadd2(and_or(w, k.even, k.magic), __float2half2_rn(-1032.f));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t code_odd(uint32_t w, const Magic& k) {
  const __half2 y = __hfma2(and_or(w, k.odd, k.magic), __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
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

// How the work is dealt out. Entry b has n_b = ceil(kv_len_b / CK) chunks; the chunks of all
// entries in a row, T of them, are cut into G = min(groups, T) ranges that differ by at most
// one chunk, whatever the lengths; a group of blocks takes a range, one block for each head
// tile (HB heads and up to 8 NT query rows), so that blocks that run side by side read
// neighbouring heads of the same tokens. (With each block's range in one head tile only, the
// copies of the full-size step alone took 473 us instead of 371.) A block finishes the entries
// that lie within its range and leaves states for the others in the workspace: slot 0 for the
// entry that began before its range, slot 1 for the one that goes on after it.
__device__ __forceinline__ int kv4_len(const DecodeKv4Args& a, int b) {
  // device-side lengths are clamped into [0, L] so a bad value cannot read past the cache
  return a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.cache.L) : a.cache.L;
}
struct Kv4Cuts {
  uint32_t each, more;  // range i has `each` chunks, and one more for i < more
  __device__ Kv4Cuts(uint32_t T, uint32_t groups) {
    const uint32_t G = min(groups, T);
    each = G ? T / G : 0;
    more = G ? T % G : 0;
  }
  __device__ uint32_t begin(uint32_t i) const { return i * each + min(i, more); }
  __device__ uint32_t range_of(uint32_t x) const {
    const uint32_t head = more * (each + 1);
    return x < head ? x / (each + 1) : more + (x - head) / each;
  }
};

// Sum of a value over the block's first `warps` warps; `buf` holds that many.
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* buf, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t sum = 0;
  for (int w = 0; w < warps; ++w) sum += buf[w];
  return sum;
}

template <int NT, int HB, Kv4Load LOAD>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 3 : 2)
    decode_kv4_split_kernel(const __grid_constant__ CUtensorMap map, DecodeKv4Args a) {
  using TL = Tile<HB>;
  constexpr int CK = TL::CK, STAGES = TL::STAGES, PITCH = TL::PITCH, ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[STAGES];  // TMA: the chunk of a stage landed
  __shared__ int readers[STAGES];    // TMA: warps that have read it
  __shared__ uint32_t bad_rows[STAGES][CK / 32];    // kTmaPaged: rows of a page outside the pool
  __shared__ int abort_flag;
  __shared__ float red[4];
  __shared__ uint32_t sums[WARPS];
  __shared__ uint32_t first[2];  // entry of the range's first chunk, chunks before that entry
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;  // fragment row (or column) and pair index
  const int hb = warp / TL::PER_HEAD, part = warp % TL::PER_HEAD;  // this warp's head and key part
  const int tiles = (a.group + ROWS - 1) / ROWS;  // of a head's query rows
  const int HQ = a.H / HB * tiles;
  const uint32_t group = blockIdx.x / HQ;
  const int tile_h = blockIdx.x % HQ;
  const int g0 = tile_h / tiles * HB, row0 = tile_h % tiles * ROWS;  // first head, first query row
  const int g = g0 + hb;

  if constexpr (LOAD != kCopy) {
    if (tid < STAGES) {
      mbar_init(&full[tid], 1);
      readers[tid] = 0;
    }
    if (tid == 0) abort_flag = 0;
    fence_barrier_init();
  }
  cudaTriggerProgrammaticLaunchCompletion();

  // this block's range and where it begins
  uint32_t T = 0;
  if (!a.kv_len) {
    T = (uint32_t)a.B * ((a.cache.L + CK - 1) / CK);
  } else {
    for (int b0 = 0; b0 < a.B; b0 += THREADS)
      T += block_sum(b0 + tid < a.B ? (kv4_len(a, b0 + tid) + CK - 1) / CK : 0, sums, WARPS);
  }
  const Kv4Cuts cuts(T, a.groups);
  uint32_t at = cuts.begin(group);  // chunk in work
  const uint32_t range_begin = at, range_end = cuts.begin(group + 1);
  if (group >= min((uint32_t)a.groups, T)) return;
  if (!a.kv_len) {
    const uint32_t n = (a.cache.L + CK - 1) / CK;
    if (tid == 0) {
      first[0] = at / n;
      first[1] = at / n * n;
    }
  } else {
    uint32_t before = 0;
    for (int b0 = 0; b0 < a.B && before <= at; b0 += THREADS) {
      const uint32_t n = b0 + tid < a.B ? (kv4_len(a, b0 + tid) + CK - 1) / CK : 0;
      uint32_t scan = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
      }
      __syncthreads();
      if (lane == 31) sums[warp] = scan;
      __syncthreads();
      scan += before;
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) scan += sums[w];
        before += sums[w];
      }
      if (scan - n <= at && at < scan) {
        first[0] = b0 + tid;
        first[1] = scan - n;
      }
    }
  }
  __syncthreads();
  int b = (int)first[0];
  uint32_t entry_begin = first[1];

  const float sl2 = 1.4426950408889634f * (a.v1 ? 0.125f : 0.08838834764831845f);  // log2(e) / sqrt(d)
  bool bad_page = false;
  uint32_t used = 0;    // chunks that went through the ring before this entry

  for (;;) {  // one entry, or what of it lies in the range, at a time
  const int kv_len = kv4_len(a, b);
  const uint32_t entry_end = entry_begin + (kv_len + CK - 1) / CK;
  const uint32_t stop = min(entry_end, range_end);
  const int n_chunks = (int)(stop - at);
  const int t0 = (int)(at - entry_begin) * CK;  // first token

  // Paged: the pages of a chunk are looked up one chunk ahead of its copies. kTmaPaged: lane i
  // holds box i's page; kCopy: lane r the byte offset of record r. -1: no key there, -2: a
  // page outside the pool. Either way the records' scales become zero, so they count as K
  // and V rows of zeros (and keys past the end get no weight at all).
  const int box_rows = LOAD == kTmaPaged ? min(1 << a.cache.page_shift, CK) : CK;
  int64_t ahead = -1;
  auto lookup = [&](int c) {
    ahead = -1;
    if constexpr (LOAD == kTmaPaged) {
      const int tok = t0 + c * CK + lane * box_rows;
      if (lane * box_rows < CK && tok < kv_len) {
        const int64_t bi = (int64_t)b * a.cache.bt_stride + (tok >> a.cache.page_shift);
        int id = -1;
        if (in_bounds(bi, 1, a.cache.ext_bt, a.cache.dev_status, a.cache.dbg_status))
          id = __ldg(a.cache.block_table + bi);
        ahead = (unsigned)id < (unsigned)a.cache.num_pages ? id : -2;
      }
    } else if constexpr (LOAD == kCopy) {
      const int tok = t0 + c * CK + part * KEYS + lane;
      if (tok < kv_len) {
        ahead = kv4_page_offset(a.cache, b, tok);
        if (ahead < 0) ahead = -2;
      }
    }
    bad_page = bad_page || ahead == -2;
  };
  // The copies of chunk c of this entry into its stage. TMA: by one warp, the first chunks by
  // warp 0, each later one by the warp that was last to read what the stage held. kCopy: each
  // warp its own records, eight lanes the 128 code bytes of one, then lane r the scales of
  // record r.
  auto load = [&](int c) {
    const uint32_t ring = used + c;
    const int s = ring % STAGES;
    uint8_t* st = smem + s * TL::STAGE_BYTES;
    if constexpr (LOAD == kCopy) {
      const int64_t head_off = (int64_t)g * a.cache.stride[2];
      auto copy = [&](int row, int64_t row_off, int piece) {
        bool ok = row_off >= 0;
        const int64_t off = (ok ? row_off : 0) + head_off + piece * 16;
        ok = ok && in_bounds(off, 16, a.cache.ext, a.cache.dev_status, a.cache.dbg_status);
        cp_async_16(st + (part * KEYS + row) * PITCH + hb * kKv4Record + piece * 16, a.cache.base + (ok ? off : 0),
                    ok ? 16u : 0u);
      };
#pragma unroll
      for (int it = 0; it < KEYS / 4; ++it) {
        const int row = it * 4 + (lane >> 3);
        copy(row, __shfl_sync(0xffffffffu, ahead, row), lane & 7);
      }
      copy(lane, ahead, 8);
    } else {
      // HB = 1: one head's records {144 bytes, head, token, entry}; else whole token rows
      const int x = HB == 1 ? 0 : g0 * (kKv4Record / 4), y = HB == 1 ? g0 : 0;
      if constexpr (LOAD == kTma) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[s], TL::STAGE_BYTES);
          tma_load_4d(st, &map, &full[s], x, y, t0 + c * CK, b);
        }
      } else {
        const uint32_t boxes = __ballot_sync(0xffffffffu, ahead >= 0);
        const uint32_t bad = __ballot_sync(0xffffffffu, ahead == -2);
        if (lane < CK / 32) {  // the bad boxes' rows, 32 to a word
          uint32_t rows = 0;
          for (int r = 0; r < 32; r += min(box_rows, 32))
            if ((bad >> ((lane * 32 + r) / box_rows)) & 1u)
              rows |= (box_rows >= 32 ? 0xffffffffu : (1u << box_rows) - 1u) << r;
          bad_rows[s][lane] = rows;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[s], __popc(boxes) * box_rows * PITCH);
        __syncwarp();
        if (ahead >= 0)
          tma_load_4d(st + lane * box_rows * PITCH, &map, &full[s], x, y,
                      (t0 + c * CK + lane * box_rows) & ((1 << a.cache.page_shift) - 1), (int)ahead);
      }
    }
  };

  constexpr int AHEAD = LOAD == kCopy ? STAGES - 1 : STAGES;  // chunks in flight or in work
  if (LOAD == kCopy || warp == 0) {
    for (int c = 0; c < AHEAD; ++c) {
      if (c < n_chunks) {
        lookup(c);
        load(c);
      }
      if constexpr (LOAD == kCopy) cp_async_commit();
    }
  }
  bool ok = true;  // no wait has run out

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
    const float down = ldexpf(sl2, 24 - 141 + max(ex, 14));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int from = (2 * tq + j) * 4;  // a lane of column 2 tq + j
      factor[nt][j] = __shfl_sync(0xffffffffu, down, from);
#pragma unroll
      for (int gr = 0; gr < 4; ++gr)
        start[nt][gr][j] = start[nt][gr][2 + j] = __shfl_sync(0xffffffffu, sums[gr], from);
    }
  }

  const Magic magic;
  // columns 2 tq, 2 tq + 1: the running maximum plus kSlack; kTop - maximum - E, twice; sums of
  // p over the keys gq and gq + 8 of each 16
  float limit[NT][2];
  float2 bias[NT][2], l[NT][2];
  float bound_E = -90.f;
  uint32_t scale_bound = 0;  // bf16 bits that no V scale so far passes, twice
  // [group][tile]: channels 32 g + 4 gq + 2 tile + {0, 1}
  float o[NT][4][2][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      limit[nt][j] = -INFINITY;
      bias[nt][j] = make_float2(0.f, 0.f);
      l[nt][j] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int gr = 0; gr < 4; ++gr)
#pragma unroll
      for (int ti = 0; ti < 2; ++ti)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][gr][ti][i] = 0.f;
  }

  lookup(AHEAD);
  for (int c = 0; c < n_chunks; ++c) {
    if constexpr (LOAD == kCopy) {
      if (c + AHEAD < n_chunks) load(c + AHEAD);
      cp_async_commit();
    }
    const uint32_t ring = used + c;
    const int stage = ring % STAGES;
    uint8_t* st = smem + stage * TL::STAGE_BYTES + part * KEYS * PITCH + hb * kKv4Record;  // this warp's records
    const int left = kv_len - (t0 + c * CK + part * KEYS);  // keys of them that exist
    if constexpr (LOAD == kCopy) {
      cp_async_wait<AHEAD>();
      __syncwarp();
    } else {
      ok = ok && mbar_wait(&full[stage], (ring / STAGES) & 1, &abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint32_t out = 0;
      if constexpr (LOAD == kTmaPaged) out = bad_rows[stage][part];
      if (left < KEYS || out) {  // scales of records that are not there
        if (lane >= left || ((out >> lane) & 1u))
          *reinterpret_cast<uint4*>(st + lane * PITCH + kKv4Scales) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();  // before a later TMA copy rewrites the stage
        __syncwarp();
      }
    }
    if (left > 0) {
    const uint32_t st32 = smem_u32(st);

    // the largest V scales of this lane's record, as magnitudes (bf16 bits are ordered)
    const uint2 vs = *reinterpret_cast<const uint2*>(st + lane * PITCH + kKv4Scales + 8);
    const uint32_t big = __vmaxu2(vs.x & 0x7fff7fffu, vs.y & 0x7fff7fffu);

    // scores of 2 x 16 keys: x[.][mt][0, 1] key mt * 16 + gq, [2, 3] key + 8, columns 2tq, +1
    float x[NT][2][4];
    uint4 scales[2][2];  // of those keys: {K 0 1, K 2 3, V 0 1, V 2 3}
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        scales[mt][h] =
            *reinterpret_cast<const uint4*>(st + (mt * 16 + h * 8 + gq) * PITCH + kKv4Scales);
      const uint32_t row = st32 + (mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * PITCH + (lane >> 4) * 16;
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

    // keys past the end get -inf; does a score or a V scale pass its bound?
    bool raise = __vmaxu2(big, scale_bound) != scale_bound;
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
        top[nt][j] = factor[nt][j] * fmaxf(fmax3(x[nt][0][j], x[nt][0][2 + j], x[nt][1][j]), x[nt][1][2 + j]);
        raise = raise || top[nt][j] > limit[nt][j];
      }
    }
    if (__any_sync(0xffffffffu, raise)) {
      // E: |scale| < 2^E for all V scales so far (not below -90, so that p does not overflow
      // over rows of zeros)
      const uint32_t most = __reduce_max_sync(0xffffffffu, max(big & 0xffffu, big >> 16));
      const float E = fmaxf((float)((int)(most >> 7) - 126), bound_E);
      bound_E = E;
      scale_bound = ((uint32_t)((int)E + 126) << 7 | 0x7fu) * 0x10001u;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float t = top[nt][j];
#pragma unroll
          for (int s = 4; s <= 16; s <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
          // what p was weighted with is `bias`, to the last bit: alpha and M go by it
          const float now = fmaxf(limit[nt][j] - kSlack, t);
          const float to = now == -INFINITY ? kTop - E : kTop - E - now;
          const float alpha = limit[nt][j] == -INFINITY ? 0.f : ex2(to - bias[nt][j].x);
          limit[nt][j] = now + kSlack;
          bias[nt][j] = make_float2(to, to);
          l[nt][j].x *= alpha;
          l[nt][j].y *= alpha;
#pragma unroll
          for (int gr = 0; gr < 4; ++gr)
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {
              o[nt][gr][ti][j] *= alpha;
              o[nt][gr][ti][2 + j] *= alpha;
            }
        }
    }
    // p of the keys (gq, gq + 8) of each 16, per column
    float2 p[NT][2][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 y = fma2(make_float2(x[nt][mt][j], x[nt][mt][2 + j]),
                                make_float2(factor[nt][j], factor[nt][j]), bias[nt][j]);
          p[nt][mt][j] = make_float2(ex2(y.x), ex2(y.y));
          l[nt][j] = add2(l[nt][j], p[nt][mt][j]);
        }

    // O += (p scale)^T-fragments times V
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t row = st32 + (mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * PITCH + kKv4VCodes + (lane >> 4) * 16;
#pragma unroll
      for (int gp = 0; gp < 2; ++gp) {
        uint32_t r[4];
        ldsm4_t(row + gp * 32, r);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const int gr = 2 * gp + gg;
          const uint32_t v0 = gp ? scales[mt][0].w : scales[mt][0].z, v1 = gp ? scales[mt][1].w : scales[mt][1].z;
          const float2 s01 = gg ? make_float2(bf16_high(v0), bf16_high(v1)) : make_float2(bf16_low(v0), bf16_low(v1));
          const uint32_t lo = r[2 * gg], hi = r[2 * gg + 1], lo8 = lo >> 8, hi8 = hi >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 w0 = mul2(p[nt][mt][0], s01), w1 = mul2(p[nt][mt][1], s01);
            const uint32_t b0 = transpose8(pack_f16(w0.x, w1.x));
            const uint32_t b1 = transpose8(pack_f16(w0.y, w1.y));
            float(&o0)[4] = o[nt][gr][0];
            float(&o1)[4] = o[nt][gr][1];
            mma_f16(o0, code_even(lo, magic), code_odd(lo, magic), code_even(hi, magic), code_odd(hi, magic), b0, b1, o0);
            mma_f16(o1, code_even(lo8, magic), code_odd(lo8, magic), code_even(hi8, magic), code_odd(hi8, magic), b0, b1, o1);
          }
        }
      }
    }
    }
    __syncwarp();  // every lane has read the stage
    if constexpr (LOAD != kCopy) {
      int last = 0;
      if (lane == 0) {
        asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(last) : "r"(smem_u32(&readers[stage])) : "memory");
        last = last == WARPS - 1;
        if (last) readers[stage] = 0;  // read next by warps that have waited for the next chunk
      }
      last = __shfl_sync(0xffffffffu, last, 0);
      if (last && c + AHEAD < n_chunks) load(c + AHEAD);
    }
    lookup(c + AHEAD + 1);
  }
  if constexpr (LOAD == kCopy) {
    cp_async_wait<0>();
  } else if (!__syncthreads_and(ok)) {
    // a copy that never landed: let the ones in flight finish before the block ends
    if (tid < STAGES) {
      const int c = n_chunks <= STAGES ? tid : n_chunks - 1 - (n_chunks - 1 - tid) % STAGES;
      if (c < n_chunks) mbar_wait_drain(&full[(used + c) % STAGES], ((used + c) / STAGES) & 1);
    }
    if (tid == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_TIMEOUT);
    break;
  }
  used += n_chunks;

  // the warps' states, [warp][row][channel] outputs and (M, l), in the ring's memory; then the
  // warps of a head joined
  float* sm_o = reinterpret_cast<float*>(smem);
  float* sm_ml = sm_o + WARPS * ROWS * W;
  static_assert(WARPS * ROWS * (W + 2) * 4 <= TL::SMEM_BYTES, "the join fits in the ring");
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = warp * ROWS + nt * 8 + 2 * tq + j;
      float sum = l[nt][j].x + l[nt][j].y;
#pragma unroll
      for (int s = 4; s <= 16; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      if (gq == 0) {
        sm_ml[2 * row] = limit[nt][j] == -INFINITY ? -INFINITY : -bias[nt][j].x;
        sm_ml[2 * row + 1] = sum;
      }
#pragma unroll
      for (int gr = 0; gr < 4; ++gr)
        *reinterpret_cast<float4*>(sm_o + row * W + gr * 32 + gq * 4) =
            make_float4(o[nt][gr][0][j], o[nt][gr][0][2 + j], o[nt][gr][1][j], o[nt][gr][1][2 + j]);
    }
  __syncthreads();
  const bool whole = entry_begin >= range_begin && entry_end <= range_end;
  const int slot = entry_begin < range_begin ? 0 : 1;
  const int rows = min(ROWS, a.group - row0);
  for (int h = 0; h < HB; ++h) {
    float prev = 0.f;
    for (int r = 0; r < rows; ++r) {
      const int from = h * TL::PER_HEAD * ROWS + r;  // the head's first warp; its others ROWS apart
      float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < TL::PER_HEAD; ++w) M = fmaxf(M, sm_ml[2 * (from + w * ROWS)]);
#pragma unroll
      for (int w = 0; w < TL::PER_HEAD; ++w) {
        const float mw = sm_ml[2 * (from + w * ROWS)];
        // a warp without keys, or with none above -inf, has M = -inf and nothing to add; only
        // a NaN among its sums is passed on
        const float f = mw == -INFINITY ? 1.f : ex2(mw - M);
        L = fmaf(sm_ml[2 * (from + w * ROWS) + 1], f, L);
        O = fmaf(sm_o[(from + w * ROWS) * W + tid], f, O);
      }
      if (whole) {
        const float y = L == 0.f ? 0.f : O / L;
        const int head = g0 + h;
        if (r & 1) store_unit(a, b, a.v1 ? head : (head * a.group + row0 + r) >> 1, tid, true, prev, y, red);
        prev = y;
      } else {
        const int64_t rec = (((int64_t)blockIdx.x * 2 + slot) * HB + h) * ROWS + r;
        if (in_bounds(rec * W + tid, 1, a.ext_ws_o, a.cache.dev_status, a.cache.dbg_status))
          a.ws_o[rec * W + tid] = O;
        if (tid == 0 && in_bounds(rec * 2, 2, a.ext_ws_ml, a.cache.dev_status, a.cache.dbg_status)) {
          a.ws_ml[rec * 2] = M;
          a.ws_ml[rec * 2 + 1] = L;
        }
      }
    }
  }
  at = stop;
  if (at == range_end) break;
  entry_begin = entry_end;
  do ++b;  // the next entry that has keys
  while (kv4_len(a, b) == 0);
  fence_proxy_async();  // the join's stores before the next entry's copies
  __syncthreads();
  }
  if (bad_page) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
}

// Joins the states of the units that several blocks share, and writes the zero rows of entries
// without keys: one block per output unit (V1 head or V2 pair) and entry. A state's weight
// 2^(M_s - M) is computed once by one thread; SLICES threads per value channel then add every
// SLICES-th state, both rows, and their sums are added in order. (With one thread per channel
// walking all states the join of 103 of them took 52 us, more than the attention.)
constexpr int SLICES = 4;
constexpr int JOIN = 128;  // states whose weights are held at a time
__global__ void __launch_bounds__(W * SLICES) decode_kv4_combine_kernel(DecodeKv4Args a) {
  __shared__ float weight[2][JOIN];
  __shared__ float part[SLICES][2][W];
  __shared__ float red[2][W * SLICES / 32];
  __shared__ uint32_t sums[W * SLICES / 32];
  constexpr int COMBINE_WARPS = W * SLICES / 32;
  const int u = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, c = tid % W, slice = tid / W;
  // the unit's head, row and head tile
  const int head = a.v1 ? u : 2 * u / a.group, row = 2 * u - head * a.group;
  const int ck = KEYS * (WARPS / a.heads), per = 8 * a.nt, tiles = (a.group + per - 1) / per;
  const int HQ = a.H / a.heads * tiles, tile_h = head / a.heads * tiles + row / per;
  const uint32_t n = (kv4_len(a, b) + ck - 1) / ck;
  uint32_t T, begin;
  if (!a.kv_len) {
    T = a.B * n;
    begin = b * n;
  } else {
    uint32_t all = 0, lower = 0;
    for (int i = tid; i < a.B; i += W * SLICES) {
      const uint32_t chunks = (kv4_len(a, i) + ck - 1) / ck;
      all += chunks;
      if (i < b) lower += chunks;
    }
    T = block_sum(all, sums, COMBINE_WARPS);
    begin = block_sum(lower, sums, COMBINE_WARPS);
  }
  const Kv4Cuts cuts(T, a.groups);
  const uint32_t i0 = n ? cuts.range_of(begin) : 0, i1 = n ? cuts.range_of(begin + n - 1) : 0;
  cudaGridDependencySynchronize();  // the split kernel's states
  if (n && i0 == i1) return;        // finished there
  // state s: slot 1 of range i0's block, then slot 0 of the ranges after it
  const int splits = n ? (int)(i1 - i0) + 1 : 0;
  const int64_t step = 2LL * HQ * a.heads * per;
  const int64_t rec0 = (((int64_t)i0 * HQ + tile_h) * 2 * a.heads + head % a.heads) * per + row % per;
  auto record = [&](int s) { return rec0 + (s ? s * step : (int64_t)a.heads * per); };
  const bool ok =
      !splits ||
      (in_bounds(record(splits - 1) * 2, 4, a.ext_ws_ml, a.cache.dev_status, a.cache.dbg_status) &&
       in_bounds(record(splits - 1) * W, 2 * W, a.ext_ws_o, a.cache.dev_status, a.cache.dbg_status));
  const int have = ok ? splits : 0;

  float M[2] = {-INFINITY, -INFINITY};
  for (int s = tid; s < have; s += W * SLICES)
#pragma unroll
    for (int e = 0; e < 2; ++e) M[e] = fmaxf(M[e], a.ws_ml[2 * (record(s) + e)]);
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
  for (int s0 = 0; s0 < have; s0 += JOIN) {
    const int held = min(JOIN, have - s0);
    __syncthreads();
    if (tid < 2 * JOIN && tid % JOIN < held) {
      const int e = tid / JOIN, s = tid % JOIN;
      const float2 v = *reinterpret_cast<const float2*>(a.ws_ml + 2 * (record(s0 + s) + e));
      // a state without keys has M = -inf and nothing to add; only a NaN is passed on
      const float f = v.x == -INFINITY ? 1.f : ex2(v.x - (e ? M[1] : M[0]));
      weight[e][s] = f;
      L = fmaf(v.y, f, L);
    }
    __syncthreads();
#pragma unroll 4
    for (int s = slice; s < held; s += SLICES) {
      const float* po = a.ws_o + record(s0 + s) * W + c;
      O[0] = fmaf(po[0], weight[0][s], O[0]);
      O[1] = fmaf(po[W], weight[1][s], O[1]);
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

// Heads of a block: neighbours read together (one run of 144 HB bytes per token) when the
// cache keeps them side by side. On the full-size step copies alone took 430 us with runs of
// 144 bytes, 390 with 288 and 371 with 576 (the cache once at 6.5 TB/s).
static int kv4_heads(int H, int64_t head_stride, bool copy) {
  if (copy || (H > 1 && head_stride != kKv4Record)) return 1;
  return H % 4 == 0 ? 4 : (H % 2 == 0 ? 2 : 1);
}

// Groups of blocks (Kv4Cuts): `num_splits` for each entry on average if that is given, else as
// many as run at once, but not so many that the chunks of full-length entries do not give each
// kMin. States are kept for two entries of every block.
void decode_kv4_plan(DecodeKv4Args* a, int num_splits) {
  constexpr int64_t kMin = 2;
  const int page = 1 << a->cache.page_shift;
  a->nt = a->group > 8 ? 2 : 1;
  a->heads = kv4_heads(a->H, a->cache.stride[2], a->cache.num_pages > 0 && page < 8);
  const int64_t ck = KEYS * (WARPS / a->heads);
  const int64_t HQ = a->H / a->heads * ((a->group + 8 * a->nt - 1) / (8 * a->nt));
  a->chunks = (int64_t)a->B * ((a->cache.L + ck - 1) / ck);
  int64_t groups = num_splits ? (int64_t)num_splits * a->B : 148 * (a->nt == 1 ? 3 : 2) / HQ;
  const int64_t most = num_splits ? a->chunks : (a->chunks + kMin - 1) / kMin;
  if (groups > most) groups = most;
  if (groups > (1 << 16)) groups = 1 << 16;
  a->groups = groups < 1 ? 1 : (int)groups;
  a->blocks = a->groups * HQ;
  a->states = a->blocks * 2 * a->heads * 8 * a->nt;
}

// HB = 1: {144 bytes, heads, rows, entries or pages}, boxes of one head's records; else
// {bytes of a token's heads, 1, rows, entries or pages}, boxes of HB heads' records and 16
// bytes (zeros behind the last head). 4-byte elements. False where TMA does not take the strides.
template <int HB>
static bool kv4_map(CUtensorMap* m, const Kv4Cache& c, int H, int rows, int outer, int box) {
  auto fn = encode_fn();
  if (!fn || rows < 1) return false;
  int64_t hs = c.stride[2], ts = c.stride[1], os = c.stride[0];
  // extents of 1 may carry any stride; give TMA a well-formed one
  if (H == 1) hs = kKv4Record;
  if (rows == 1) ts = hs * H;
  if (outer == 1) os = ts * rows;
  const int inner = HB == 1 ? kKv4Record / 4 : H * (kKv4Record / 4);
  if (HB != 1) hs = (int64_t)inner * 4;
  const cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)(HB == 1 ? H : 1), (cuuint64_t)rows, (cuuint64_t)outer};
  const cuuint64_t strides[3] = {(cuuint64_t)hs, (cuuint64_t)ts, (cuuint64_t)os};
  const cuuint32_t boxes[4] = {(cuuint32_t)Tile<HB>::PITCH / 4, 1, (cuuint32_t)box, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, c.base, dims, strides, boxes, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, int HB>
static cudaError_t launch_split(const DecodeKv4Args& a, cudaStream_t stream) {
  using TL = Tile<HB>;
  const bool paged = a.cache.block_table != nullptr;
  const int page = 1 << a.cache.page_shift;
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  Kv4Load how = kCopy;
  if (!paged && kv4_map<HB>(&map, a.cache, a.H, a.cache.L, a.B, TL::CK)) how = kTma;
  if (paged && page >= 8 &&
      kv4_map<HB>(&map, a.cache, a.H, page, a.cache.num_pages, page < TL::CK ? page : TL::CK))
    how = kTmaPaged;
  void (*const fns[3])(CUtensorMap, DecodeKv4Args) = {decode_kv4_split_kernel<NT, HB, kTma>,
                                                      decode_kv4_split_kernel<NT, HB, kTmaPaged>,
                                                      decode_kv4_split_kernel<NT, HB, kCopy>};
  void (*const fn)(CUtensorMap, DecodeKv4Args) = fns[how];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool attr_set[3][64] = {};
  if (dev >= 64 || !attr_set[how][dev]) {
    e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, TL::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[how][dev] = true;
  }
  fn<<<(unsigned)a.blocks, THREADS, TL::SMEM_BYTES, stream>>>(map, a);
  return cudaGetLastError();
}

cudaError_t launch_decode_kv4(const DecodeKv4Args& a, cudaStream_t stream) {
  cudaError_t e;
  if (a.nt == 1)
    e = a.heads == 4 ? launch_split<1, 4>(a, stream) : (a.heads == 2 ? launch_split<1, 2>(a, stream) : launch_split<1, 1>(a, stream));
  else
    e = a.heads == 4 ? launch_split<2, 4>(a, stream) : (a.heads == 2 ? launch_split<2, 2>(a, stream) : launch_split<2, 1>(a, stream));
  if (e != cudaSuccess) return e;
  // launched while the last blocks still run; the kernel waits for them itself
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
