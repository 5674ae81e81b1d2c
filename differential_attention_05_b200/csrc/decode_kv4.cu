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
// A block takes up to four neighbouring KV heads and a run of tokens; one warp issues the
// copies into a ring of stages, the others compute, each with 32 keys of a head at a time and
// its own running maximum, sums and output; a second kernel joins what several blocks did of
// an entry. Products run on mma.sync m16n8k16 in fp16 with fp32 sums, keys (or value
// channels) as the 16 rows and query rows as the 8 columns:
//   * Codes go from shared memory to registers by ldmatrix (keys: one 16-byte group of a row
//     per matrix row, a thread gets 8 channels of one key; values: transposed, a thread gets
//     4 channels of two neighbouring keys, which is the pair an MMA operand register holds).
//   * K nibbles are used as fp16 subnormals: n in the low mantissa bits is n 2^-24, the next
//     nibble 16 n 2^-24 against q / 16, so unpacking is one AND for two channels. The -8 comes
//     in as a product of the scales and -8 * 2^-24 sum q (in three bf16 parts), one MMA for 16
//     keys, from which the scores start: half the range is all that cancels.
//   * V nibbles become n - 8 exactly (0x6400 | n is 1024 + n). Left as subnormals with the -8
//     from a second MMA over constants the full step took 3% less, but the
//     cancelling sums lost up to 2^-16 of a scale, which shows where a peaked row's key has
//     the code 0.
//   * Scales stay outside the MMAs: a group is two k-steps, its fp32 sums are scaled and
//     added; for V the probability is multiplied by the scale in fp32 and rounded to fp16
//     once (2^-11 relative; bf16's 2^-8 would be amplified by the subtraction and V1's norm).
//     fp16's range is kept by the running maximum M of the scores and the exponent E of the
//     largest V scale so far: p = 2^(x - M), and the operand is p 2^(kTop - E) times the scale,
//     under 2^(kTop + kSlack). M is raised only when a score passes it by kSlack. The largest
//     scale is 2^(E - 1) or more, so the largest probability times it makes an operand of 2^8 or
//     more, and products under 2^-22 of that become subnormal and lose bits.
//     M and the sums of p follow the scores alone. (With 2^(kTop - E) as a part of p, which saves
//     four instructions a chunk, a V scale 2^36 times those before it made all their
//     probabilities flush to 0, in the sums too: 32 keys of V = 0 counted for nothing.)
//   * The branches' rounding errors do not cancel in O_1 / l_1 - lambda O_2 / l_2, while the
//     values may: with lambda near 1 and flat scores (V1's norm then scales the rest up) the
//     output was 0.0027 off in relative terms where its bf16 rounding alone makes 0.0016. So
//     the operand of branch 1 is p_1 - c p_2, formed in fp32: D = O_1 - c O_2 carries errors of
//     its own size only, those of O_2 cancel as far as c is near lambda l_1 / l_2, and
//     O_1 = D + c O_2 is put together in fp32 when the warp is done. c is that ratio of the
//     sums so far (0 to 1), but no larger than keeps c p_2 <= 1.25 p_1 for every key that meets
//     it. That is what makes it safe: a key's rounding errors then move the output by at most
//     2^-11 (|p_1 - c p_2| / l_1 + |c / l_1 - lambda / l_2| p_2) <= 2^-11 (1.5 p_1 / l_1 +
//     |lambda| p_2 / l_2) times its |v|, where c = 0 has 1 for the 1.5. (The room of 1.25 leaves
//     c alone under flat scores: with 1, V1's error at lambda = 1 was 0.0021, not 0.0017. Held by the sums alone, at every
//     fourth chunk, c let a branch 2 that rises behind a sink of both put errors of c p_2 into D
//     that are many times O_1's own: 0.009 to 0.09 of the output.) Both branches of a unit are
//     neighbouring columns of one lane, so this costs a dozen instructions a chunk (467 us for
//     447 on the full step).
//   * q is taken times a power of two per row so that its largest element is in [2^14, 2^15);
//     fp16 then holds elements above 2^-31 of the largest exactly in even channels, and above
//     2^-27 in odd ones, which are divided by 16.
//
// What bounds it: power, then issue slots. V2, 64 entries x 32768 tokens x 8 heads (2.42 GB, 374
// us at the copy rate): 469 us alone, 510 to 550 us call after call, when the GPU holds its 1000
// W at 1690 MHz. 32 keys of a head are about 540 warp instructions, 224 of them unpacking; with
// the data in L2 the same loop took no less. V1, 32 x 32768 x 16: 463 us alone, 522 at 1730 MHz.
#include <cuda_fp16.h>

#include <string.h>

#include "kv4.cuh"
#include "tma_host.cuh"

namespace diffattn {

namespace {
constexpr int W = kKv4Width;
constexpr int KEYS = 32;      // keys that a warp takes of a chunk
constexpr int kTop = 9;       // p * scale < 2^kTop in units of 2^E when the maximum is raised ...
constexpr float kSlack = 6.f; // ... and < 2^(kTop + kSlack) before, inside fp16's range: |p_1 - c p_2| <= p_1
constexpr int kLeastE = -102; // the exponent E of the V scales: scales that are held are 2^-103 and more
constexpr float kRoom = 0.32192809f;  // log2(1.25): c p_2 <= 1.25 p_1
constexpr float kJoin = 1.f / (1 << 30) / 64.f;  // see the join's weights

// A block has CW warps that compute and one that issues the copies; three blocks to an SM.
constexpr int CW = 4;
constexpr int THREADS = (CW + 1) * 32;
constexpr int ROWS = 8;       // query rows of a block, the columns of its MMAs
constexpr int kBlocksPerSm = 3;

// A block takes HB neighbouring KV heads, CW / HB warps for each. A chunk is CK tokens in a
// stage of one row per token: the HB records side by side, as they lie in the cache, and 16
// bytes more (of the next record, unused) where that is needed for a pitch that is an odd
// number of 16-byte units, so that ldmatrix's 8 rows meet no bank twice.
template <int HB>
struct Tile {
  static constexpr int PER_HEAD = CW / HB;  // warps of a head
  static constexpr int CK = KEYS * PER_HEAD;
  static constexpr int PITCH = HB * kKv4Record + (HB == 1 ? 0 : 16);
  static constexpr int STAGE_BYTES = CK * PITCH;
  // what shared memory holds beside the states that the warps of a head join at the end
  static constexpr int STAGES = HB == 4 ? 4 : 3;
  static constexpr int JOIN_FLOATS = (PER_HEAD - 1) * HB * ROWS * (W + 2);
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + JOIN_FLOATS * 4;
  static_assert((PITCH / 16) % 2 == 1 && STAGE_BYTES % 128 == 0 && 8 * PITCH % 128 == 0, "layout");
  static_assert(kBlocksPerSm * (SMEM_BYTES + 2048) <= 228 * 1024, "shared memory");
};

// How a chunk reaches shared memory: TMA boxes of CK rows (contiguous) or of a page's run of
// up to CK (pages of 8 tokens and more; a box of fewer would not end on a 128-byte boundary),
// or one bulk copy for each token (smaller pages, and strides that TMA does not take).
enum Kv4Load { kTma, kTmaPaged, kRows };
}  // namespace

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// d = a b + c; mma_f16 without c and mma_bf16: d = a b
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
// 2^(kTop - E) from a pair of bounds (E + 126) << 7 | 0x7f on the V scales' bf16 bits
__device__ __forceinline__ float kv4_unit(uint32_t scale_bound) {
  return __uint_as_float((uint32_t)(127 + kTop + 126 - (int)(scale_bound >> 23)) << 23);
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

// How the work is dealt out. Entry b has n_b = ceil(kv_len_b / CK) chunks; the chunks of all
// entries in a row, T of them, are cut into G = min(groups, T) ranges that differ by at most
// one chunk, whatever the lengths; a group of blocks takes a range, one block for each head
// tile (HB heads and up to 8 query rows of each), so that blocks that run side by side read
// neighbouring heads of the same tokens. (More than 8 query rows to a head take another tile,
// which reads the records again, mostly from L2. With 16 rows in a block the accumulators left
// one block of 8 warps to an SM: 16 rows over 32 x 8192 tokens x 2 heads took 57 us, not 43.) (With each block's range in one head tile only, the
// copies of the full-size step alone took 473 us instead of 371.) A block finishes the entries
// that lie within its range and leaves states for the others in the workspace: slot 0 for the
// entry that began before its range, slot 1 for the one that goes on after it.
// Short entries (by_entry) go whole to a group each, which needs no scan, no workspace and no
// second kernel.
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

// The consumers' barrier (the copying warp does not take part).
template <int THREADS>
__device__ __forceinline__ void bar_consumers() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

template <int HB, Kv4Load LOAD>
__global__ void __launch_bounds__(THREADS, kBlocksPerSm)
    decode_kv4_split_kernel(const __grid_constant__ CUtensorMap map, DecodeKv4Args a) {
  using TL = Tile<HB>;
  constexpr int CK = TL::CK, STAGES = TL::STAGES, PITCH = TL::PITCH, WARPS = CW + 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[STAGES], empty[STAGES];  // the chunk of a stage has landed; was read
  __shared__ uint32_t bad_rows[STAGES][CK / 32];    // rows of a chunk of a page outside the pool
  __shared__ int abort_flag;
  __shared__ uint32_t sums[WARPS];
  __shared__ uint32_t first[2];  // entry of the range's first chunk, chunks before that entry
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (a.group + ROWS - 1) / ROWS;  // of a head's query rows
  const int HQ = a.H / HB * tiles;
  const uint32_t group = blockIdx.x / HQ;
  const int tile_h = blockIdx.x % HQ;
  const int g0 = tile_h / tiles * HB, row0 = tile_h % tiles * ROWS;  // first head, first query row

  if (tid < STAGES) {
    mbar_init(&full[tid], 1);
    mbar_init(&empty[tid], CW);
  }
  if (tid == 0) abort_flag = 0;
  fence_barrier_init();
  cudaTriggerProgrammaticLaunchCompletion();  // the join may be launched

  int b = (int)group;
  uint32_t range_begin = 0, range_end, entry_begin = 0;
  if (a.by_entry) {
    range_end = (kv4_len(a, b) + CK - 1) / CK;
    __syncthreads();
    if (range_end == 0) {  // no key: zeros
      const int units = a.v1 ? 1 : min(ROWS, a.group - row0) / 2;
      for (int i = tid; i < HB * units * W; i += THREADS) {
        const int head = g0 + i / (units * W), unit = i / W % units;
        const int64_t off = b * a.os[0] + (int64_t)(a.v1 ? head : (head * a.group + row0) / 2 + unit) * a.os[1] + i % W;
        if (in_bounds(off, 1, a.ext_out, a.cache.dev_status, a.cache.dbg_status))
          static_cast<__nv_bfloat16*>(a.out)[off] = __float2bfloat16_rn(0.f);
      }
      return;
    }
  } else {
    // this block's range and where it begins: chunks of the entries before each (`scan`, of
    // THREADS entries at a time)
    uint32_t T = 0, n = 0, scan = 0;
    auto scan_entries = [&](int b0, uint32_t before) {  // returns the chunks up to their end
      n = b0 + tid < a.B ? (kv4_len(a, b0 + tid) + CK - 1) / CK : 0;
      scan = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
      }
      if (lane == 31) sums[warp] = scan;
      __syncthreads();
      scan += before;
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) scan += sums[w];
        before += sums[w];
      }
      __syncthreads();
      return before;
    };
    if (!a.kv_len) {
      n = (a.cache.L + CK - 1) / CK;
      T = (uint32_t)a.B * n;
    } else {
      for (int b0 = 0; b0 < a.B; b0 += THREADS) T = scan_entries(b0, T);
    }
    const Kv4Cuts cuts(T, a.groups);
    range_begin = cuts.begin(group);
    range_end = cuts.begin(group + 1);
    if (group >= min((uint32_t)a.groups, T)) return;
    if (!a.kv_len) {
      if (tid == 0) {
        first[0] = range_begin / n;
        first[1] = range_begin / n * n;
      }
    } else {
      uint32_t before = 0;
      for (int b0 = 0; b0 < a.B && before <= range_begin; b0 += THREADS) {
        before = a.B <= THREADS ? T : scan_entries(b0, before);
        if (scan - n <= range_begin && range_begin < scan) {
          first[0] = b0 + tid;
          first[1] = scan - n;
        }
      }
    }
    __syncthreads();
    b = (int)first[0];
    entry_begin = first[1];
  }
  uint32_t at = range_begin;  // chunk in work
  int stage = 0;
  uint32_t parity = 0;  // of the ring's current round
  auto advance = [&] {
    if (++stage == STAGES) {
      stage = 0;
      parity ^= 1u;
    }
  };

  if (warp == CW) {
    // ---- copies: chunk after chunk of the range, through all its entries, as stages are freed
    uint32_t issued = 0;
    bool ok = true, bad_page = false;
    while (ok && at < range_end) {
      const int kv_len = kv4_len(a, b);
      const uint32_t entry_end = entry_begin + (kv_len + CK - 1) / CK, stop = min(entry_end, range_end);
      for (; ok && at < stop; ++at) {
        const int tok0 = (int)(at - entry_begin) * CK;
        uint8_t* st = smem + stage * TL::STAGE_BYTES;
        const int x = HB == 1 ? 0 : g0 * (kKv4Record / 4), y = HB == 1 ? g0 : 0;  // TMA: see kv4_map
        // The pages first, while the stage may still be in use. Rows of a page outside the pool
        // are marked and left out: their scales become zero, so they count as K and V of zeros.
        [[maybe_unused]] const int box_rows = LOAD == kTmaPaged ? min(1 << a.cache.page_shift, CK) : CK;
        [[maybe_unused]] int page = -1;
        [[maybe_unused]] int64_t off[CK / 32];
        [[maybe_unused]] uint32_t bad = 0;
        if constexpr (LOAD == kTmaPaged) {
          const int tok = tok0 + lane * box_rows;
          const bool need = lane * box_rows < CK && tok < kv_len;
          if (need) {
            const int64_t bi = (int64_t)b * a.cache.bt_stride + (tok >> a.cache.page_shift);
            if (in_bounds(bi, 1, a.cache.ext_bt, a.cache.dev_status, a.cache.dbg_status))
              page = __ldg(a.cache.block_table + bi);
            if ((unsigned)page >= (unsigned)a.cache.num_pages) page = -1;
          }
          bad = __ballot_sync(0xffffffffu, need && page < 0);
          bad_page = bad_page || bad != 0;
        } else if constexpr (LOAD == kRows) {
#pragma unroll
          for (int i = 0; i < CK / 32; ++i) {
            const int tok = tok0 + i * 32 + lane;
            off[i] = tok < kv_len ? kv4_page_offset(a.cache, b, tok) : -2;
            bad_page = bad_page || off[i] == -1;
            if (off[i] >= 0) {
              off[i] += (int64_t)g0 * a.cache.stride[2];
              if (!in_bounds(off[i], HB * kKv4Record, a.cache.ext, a.cache.dev_status, a.cache.dbg_status)) off[i] = -1;
            }
          }
        }
        if (issued >= (uint32_t)STAGES) {
          ok = mbar_wait(&empty[stage], parity ^ 1u, &abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        // Not more than two chunks on their way: at the start all blocks would otherwise ask for a
        // ring each, 34 MB, and the first chunk come in with the last (8 us into a ragged batch
        // that the last block ended at 35; now 6 and 33)
        if (issued >= 2) {
          ok = mbar_wait(&full[(issued - 2) % STAGES], ((issued - 2) / STAGES) & 1u, &abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if constexpr (LOAD == kTma) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[stage], TL::STAGE_BYTES);
            tma_load_4d(st, &map, &full[stage], x, y, tok0, b);
          }
        } else if constexpr (LOAD == kTmaPaged) {
          const uint32_t boxes = __ballot_sync(0xffffffffu, page >= 0);
          if (lane < CK / 32) {  // the bad boxes' rows, 32 to a word
            uint32_t rows = 0;
            for (int r = 0; bad && r < 32; r += min(box_rows, 32))
              if ((bad >> ((lane * 32 + r) / box_rows)) & 1u)
                rows |= (box_rows >= 32 ? 0xffffffffu : (1u << box_rows) - 1u) << r;
            bad_rows[stage][lane] = rows;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&full[stage], __popc(boxes) * box_rows * PITCH);
          __syncwarp();
          if (page >= 0)
            tma_load_4d(st + lane * box_rows * PITCH, &map, &full[stage], x, y,
                        (tok0 + lane * box_rows) & ((1 << a.cache.page_shift) - 1), page);
        } else {
          int rows = 0;
#pragma unroll
          for (int i = 0; i < CK / 32; ++i) {
            rows += __popc(__ballot_sync(0xffffffffu, off[i] >= 0));
            const uint32_t lost = __ballot_sync(0xffffffffu, off[i] == -1);
            if (lane == 0) bad_rows[stage][i] = lost;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&full[stage], rows * HB * kKv4Record);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < CK / 32; ++i)
            if (off[i] >= 0) bulk_load(st + (i * 32 + lane) * PITCH, a.cache.base + off[i], HB * kKv4Record, &full[stage]);
        }
        ++issued;
        advance();
      }
      if (ok && at < range_end) {
        entry_begin = entry_end;
        do ++b;  // the next entry that has keys
        while (kv4_len(a, b) == 0);
      }
    }
    if (bad_page) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
    if (!ok) {
      // the readers gave up: the copies in flight end before the block does
      const uint32_t from = issued > (uint32_t)STAGES ? issued - STAGES : 0;
      for (uint32_t i = from; i < issued; ++i) mbar_wait_drain(&full[i % STAGES], (i / STAGES) & 1u);
    }
    return;
  }

  // ---- compute
  const int gq = lane >> 2, tq = lane & 3;  // fragment row (or column) and pair index
  const int hb = warp / TL::PER_HEAD, part = warp % TL::PER_HEAD;  // this warp's head and key part
  const int g = g0 + hb;
  const float sl2 = 1.4426950408889634f * (a.v1 ? 0.125f : 0.08838834764831845f);  // log2(e) / sqrt(d)
  const Magic magic;
  bool ok = true;  // no wait has run out

  for (;;) {  // one entry, or what of it lies in the range, at a time
    const int kv_len = kv4_len(a, b);
    const uint32_t entry_end = entry_begin + (kv_len + CK - 1) / CK, stop = min(entry_end, range_end);

    // Query fragments (B operands), rows scaled to fp16: for group gr and k-step ks, register 0
    // holds channels 32 gr + 8 tq + 2 ks + {0, 4}, register 1 the next pair over 16 (the order
    // in which the nibbles of a word come). Lane column gq; factor is per column of the
    // accumulators, 2 tq and 2 tq + 1.
    uint32_t qb[8][2];
    uint32_t shift[2];  // the -8 of all nibbles, see the scores below
    float factor[2];    // accumulated score -> log2 domain
    const int row = row0 + gq;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    int64_t off = b * a.qs[0];
    if (a.v1) off += (int64_t)g * a.qs[1];  // the branches lie side by side in the head's row
    else off += ((int64_t)g * a.group + row) * a.qs[1];
    const bool have = row < a.group && in_bounds(off, W, a.ext_q, a.cache.dev_status, a.cache.dbg_status);
    uint4 w[4];
    float top = 0.f;
    bool odd = false;  // an infinity or a NaN
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
      // V1: row 0 has only groups 0, 1 (branch 1), row 1 only groups 2, 3 (branch 2)
      const bool mine = have && (!a.v1 || (gr >> 1) == row);
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
    float sums_q[4];  // -8 * 2^-24 * sum of the group's q
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
        qb[2 * gr + ks][0] = pack_f16(v[2 * ks], v[2 * ks + 4]);
        qb[2 * gr + ks][1] = pack_f16(v[2 * ks + 1] * 0.0625f, v[2 * ks + 5] * 0.0625f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sums_q[gr] = sum * (-8.f / 16777216.f);
    }
    // those sums in three bf16 parts (24 bits): k = 4 part + group of a B operand
    const float c0 = tq & 1 ? sums_q[2] : sums_q[0], c1 = tq & 1 ? sums_q[3] : sums_q[1];
    const uint32_t part1 = pack_bf16(c0, c1);
    const float d0 = c0 - bf16_low(part1), d1 = c1 - bf16_high(part1);
    const uint32_t part2 = pack_bf16(d0, d1);
    const uint32_t part3 = pack_bf16(d0 - bf16_low(part2), d1 - bf16_high(part2));
    shift[0] = tq < 2 ? part1 : part2;
    shift[1] = tq < 2 ? part3 : 0u;
    // 2^24 (nibbles as 2^-24) * 2^(ex - 141) * log2(e) / sqrt(d). Rows with elements past
    // 2^117 overflow here to infinite scores
    const float down = ldexpf(sl2, 24 - 141 + max(ex, 14));
#pragma unroll
    for (int j = 0; j < 2; ++j) factor[j] = __shfl_sync(0xffffffffu, down, (2 * tq + j) * 4);

    // columns 2 tq, 2 tq + 1: the running maximum plus kSlack; minus the maximum, twice; sums of
    // p over the keys gq and gq + 8 of each 16
    float limit[2];
    float2 bias[2], l[2];
    uint32_t scale_bound = ((kLeastE + 126) << 7 | 0x7f) * 0x10001u;  // bf16 bits that no V scale so far passes, twice
    float unit = kv4_unit(scale_bound);
    const bool is_unit = row0 + 2 * tq < a.group;  // columns 2 tq, 2 tq + 1: the branches of unit u
    const int u = a.v1 ? g : (g * a.group + row0 + 2 * tq) >> 1;
    const float lam = is_unit ? __ldg(a.lambda + u) : 0.f;
    float c = 0.f;            // column 2 tq accumulates p_1 - c p_2, c >= 0
    float c_room = INFINITY;  // kRoom - log2(c): c p_2 <= 1.25 p_1 for keys with log2(p_2 / p_1) up to here
    // [group][tile]: channels 32 g + 4 gq + 2 tile + {0, 1}; elements 0, 2 column 2 tq, 1, 3 the next
    float o[4][2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      limit[j] = -INFINITY;
      bias[j] = make_float2(0.f, 0.f);
      l[j] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int gr = 0; gr < 4; ++gr)
#pragma unroll
      for (int ti = 0; ti < 2; ++ti)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[gr][ti][i] = 0.f;

    int left = kv_len - (int)(at - entry_begin) * CK - part * KEYS;  // keys from this warp's first on
    uint32_t look = at;  // the chunk at which c next goes by the sums
    for (uint32_t chunk = at; chunk < stop; ++chunk, left -= CK) {
      if (ok) {
        ok = mbar_wait(&full[stage], parity, &abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_TIMEOUT);
      }
      if (ok && left > 0) {
        uint8_t* st = smem + stage * TL::STAGE_BYTES + part * KEYS * PITCH + hb * kKv4Record;  // this warp's records
        uint32_t lost = 0;
        if constexpr (LOAD != kTma) lost = bad_rows[stage][part];
        if (left < KEYS || lost) {  // scales of records that are not there
          if (lane >= left || ((lost >> lane) & 1u))
            *reinterpret_cast<uint4*>(st + lane * PITCH + kKv4Scales) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async();  // before a later copy rewrites the stage
          __syncwarp();
        }
        const uint32_t st32 = smem_u32(st) + (((lane >> 3) & 1) * 8 + (lane & 7)) * PITCH + (lane >> 4) * 16;

        // the largest V scales of this lane's record, as magnitudes (bf16 bits are ordered)
        const uint2 vs = *reinterpret_cast<const uint2*>(st + lane * PITCH + kKv4Scales + 8);
        const uint32_t big = __vmaxu2(vs.x & 0x7fff7fffu, vs.y & 0x7fff7fffu);

        // scores of 2 x 16 keys: x[.][mt][0, 1] key mt * 16 + gq, [2, 3] key + 8, columns 2tq, +1
        float x[2][4];
        // scales of those keys, {groups 0 1, 2 3}
        uint2 ks[2][2], vscale[2][2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 both = *reinterpret_cast<const uint4*>(st + (mt * 16 + h * 8 + gq) * PITCH + kKv4Scales);
            ks[mt][h] = make_uint2(both.x, both.y);
            vscale[mt][h] = make_uint2(both.z, both.w);
          }
          // sum over groups of scale * (-8 sum q), as a product of the scales and `shift`
          const uint32_t k0 = tq & 1 ? ks[mt][0].y : ks[mt][0].x;
          const uint32_t k1 = tq & 1 ? ks[mt][1].y : ks[mt][1].x;
          mma_bf16(x[mt], k0, k1, k0, k1, shift[0], shift[1]);
#pragma unroll
          for (int gp = 0; gp < 2; ++gp) {
            uint32_t r[4];
            ldsm4(st32 + mt * 16 * PITCH + gp * 32, r);
#pragma unroll
            for (int gg = 0; gg < 2; ++gg) {
              const int gr = 2 * gp + gg;
              const uint32_t lo = r[2 * gg], hi = r[2 * gg + 1], lo8 = lo >> 8, hi8 = hi >> 8;
              const uint32_t w0 = gp ? ks[mt][0].y : ks[mt][0].x, w1 = gp ? ks[mt][1].y : ks[mt][1].x;
              const float s0 = gg ? bf16_high(w0) : bf16_low(w0), s1 = gg ? bf16_high(w1) : bf16_low(w1);
              float acc[4];
              mma_f16(acc, nib_even(lo), nib_even(hi), nib_odd(lo), nib_odd(hi), qb[2 * gr][0],
                      qb[2 * gr][1]);
              mma_f16(acc, nib_even(lo8), nib_even(hi8), nib_odd(lo8), nib_odd(hi8), qb[2 * gr + 1][0],
                      qb[2 * gr + 1][1], acc);
              float* xx = x[mt];
              xx[0] = fmaf(s0, acc[0], xx[0]); xx[1] = fmaf(s0, acc[1], xx[1]);
              xx[2] = fmaf(s1, acc[2], xx[2]); xx[3] = fmaf(s1, acc[3], xx[3]);
            }
          }
        }

        // keys past the end get -inf; does a score or a V scale pass its bound?
        bool raise = __vmaxu2(big, scale_bound) != scale_bound;
        float top[2];
        if (left < KEYS) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (mt * 16 + (i >> 1) * 8 + gq >= left) x[mt][i] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[j] = factor[j] * fmaxf(fmax3(x[0][j], x[0][2 + j], x[1][j]), x[1][2 + j]);
          raise = raise || top[j] > limit[j];
        }
        if (__any_sync(0xffffffffu, raise)) {
          // |scale| < 2^E for all finite V scales so far; `shrink` is 2^(E - new E). A NaN's (or
          // an infinity's) own group is lost whatever E is, and the others' products go by theirs.
          const uint2 all = *reinterpret_cast<const uint2*>(st + lane * PITCH + kKv4Scales + 8);
          const uint32_t a0 = all.x & 0x7fff7fffu, a1 = all.y & 0x7fff7fffu;
          const uint32_t held = __vmaxu2(a0 & __vcmpltu2(a0, 0x7f807f80u), a1 & __vcmpltu2(a1, 0x7f807f80u));
          const uint32_t most = __reduce_max_sync(0xffffffffu, max(held & 0xffffu, held >> 16));
          const uint32_t was = scale_bound >> 23, now_E = max(most >> 7, was);  // E + 126
          const float shrink = __uint_as_float((uint32_t)max(127 + (int)was - (int)now_E, 0) << 23);
          scale_bound = (now_E << 7 | 0x7fu) * 0x10001u;
          unit = kv4_unit(scale_bound);
          float alpha[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float t = top[j];
#pragma unroll
            for (int s = 4; s <= 16; s <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
            // what p was weighted with is `bias`, to the last bit: alpha and M go by it
            const float now = fmaxf(limit[j] - kSlack, t);
            const float to = now == -INFINITY ? 0.f : -now;
            alpha[j] = limit[j] == -INFINITY ? 0.f : ex2(to - bias[j].x);
            limit[j] = now + kSlack;
            bias[j] = make_float2(to, to);
            l[j].x *= alpha[j];
            l[j].y *= alpha[j];
          }
          // D <- alpha_1 (D + c O_2) - c' alpha_2 O_2, O_2 <- alpha_2 O_2, c' for the new maxima
          const bool both = alpha[0] > 0.f && alpha[1] > 0.f;
          const float next = both ? fminf(__fmul_rn(c, __fdiv_rn(alpha[0], alpha[1])), 1.f) : 0.f;
          const float back = (__fmul_rn(alpha[0], c) - __fmul_rn(next, alpha[1])) * shrink;
          c = next;
          c_room = kRoom - __log2f(c);
          alpha[0] *= shrink;
          alpha[1] *= shrink;
#pragma unroll
          for (int gr = 0; gr < 4; ++gr)
#pragma unroll
            for (int ti = 0; ti < 2; ++ti)
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                o[gr][ti][i] = fmaf(back, o[gr][ti][i + 1], __fmul_rn(alpha[0], o[gr][ti][i]));
                o[gr][ti][i + 1] *= alpha[1];
              }
        }
        // p of the keys (gq, gq + 8) of each 16, per column, and the most of log2 (p_2 / p_1). (A
        // NaN, as of two scores of -inf past the end, counts for nothing in that.)
        float2 p[2][2];
        float apart = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float2 y[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            y[j] = fma2(make_float2(x[mt][j], x[mt][2 + j]), make_float2(factor[j], factor[j]), bias[j]);
            p[mt][j] = make_float2(ex2(y[j].x), ex2(y[j].y));
            l[j] = add2(l[j], p[mt][j]);
          }
          apart = fmaxf(apart, fmaxf(y[1].x - y[0].x, y[1].y - y[0].y));
        }
        // c is lambda l_1 / l_2 by the sums at chunks 1, 4, 16, ..., and made smaller before the
        // operand is formed wherever a key's c p_2 would pass 1.25 p_1, with a quarter of the
        // distance to spare so that the next such key is rare (scattered scores: some 20 times in 295 chunks; 68
        // without that and with a look at the sums at 1, 2, 4, 8, ...)
        const bool by_sums = chunk == look;
        if (by_sums || __any_sync(0xffffffffu, apart > c_room)) {
#pragma unroll
          for (int s = 4; s <= 16; s <<= 1) apart = fmaxf(apart, __shfl_xor_sync(0xffffffffu, apart, s));
          float next = c;
          if (by_sums) {
            look = at + 4 * (look - at) + 3;
            float s1 = l[0].x + l[0].y, s2 = l[1].x + l[1].y;
#pragma unroll
            for (int s = 4; s <= 16; s <<= 1) {
              s1 += __shfl_xor_sync(0xffffffffu, s1, s);
              s2 += __shfl_xor_sync(0xffffffffu, s2, s);
            }
            next = s2 > 0.f ? fminf(fmaxf(__fmul_rn(lam, __fdiv_rn(s1, s2)), 0.f), 1.f) : 0.f;
            c_room = kRoom - __log2f(next);
          }
          if (apart > c_room) {
            next = ex2(-1.25f * apart);
            c_room = fmaf(1.25f, apart, kRoom);
          }
          const float back = c - next;
          c = next;
#pragma unroll
          for (int gr = 0; gr < 4; ++gr)
#pragma unroll
            for (int ti = 0; ti < 2; ++ti)
#pragma unroll
              for (int i = 0; i < 4; i += 2) o[gr][ti][i] = fmaf(back, o[gr][ti][i + 1], o[gr][ti][i]);
        }
        // the operand of column 2 tq, see c; from here on in units of the V scales
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          p[mt][0] = mul2(fma2(p[mt][1], make_float2(-c, -c), p[mt][0]), make_float2(unit, unit));
          p[mt][1] = mul2(p[mt][1], make_float2(unit, unit));
        }

        // O += (p scale)^T-fragments times V
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int gp = 0; gp < 2; ++gp) {
            uint32_t r[4];
            ldsm4_t(st32 + kKv4VCodes + mt * 16 * PITCH + gp * 32, r);
#pragma unroll
            for (int gg = 0; gg < 2; ++gg) {
              const int gr = 2 * gp + gg;
              const uint32_t w0 = gp ? vscale[mt][0].y : vscale[mt][0].x, w1 = gp ? vscale[mt][1].y : vscale[mt][1].x;
              const float2 s01 = gg ? make_float2(bf16_high(w0), bf16_high(w1)) : make_float2(bf16_low(w0), bf16_low(w1));
              const uint32_t lo = r[2 * gg], hi = r[2 * gg + 1], lo8 = lo >> 8, hi8 = hi >> 8;
              const uint32_t a0 = code_even(lo, magic), a1 = code_odd(lo, magic), a2 = code_even(hi, magic),
                             a3 = code_odd(hi, magic);
              const uint32_t a4 = code_even(lo8, magic), a5 = code_odd(lo8, magic), a6 = code_even(hi8, magic),
                             a7 = code_odd(hi8, magic);
              const float2 p0 = mul2(p[mt][0], s01), p1 = mul2(p[mt][1], s01);
              const uint32_t b0 = transpose8(pack_f16(p0.x, p1.x));
              const uint32_t b1 = transpose8(pack_f16(p0.y, p1.y));
              mma_f16(o[gr][0], a0, a1, a2, a3, b0, b1, o[gr][0]);
              mma_f16(o[gr][1], a4, a5, a6, a7, b0, b1, o[gr][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (lane == 0) mbar_arrive(&empty[stage]);
      advance();
    }
    // The state of the warp's keys: M = -bias (-inf without a key), the sum L of p, and O / L, which
    // has the size of V whatever the sizes of the states that it will be joined with.
    float L[2], M[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      L[j] = l[j].x + l[j].y;
#pragma unroll
      for (int s = 4; s <= 16; s <<= 1) L[j] += __shfl_xor_sync(0xffffffffu, L[j], s);
      M[j] = limit[j] == -INFINITY ? -INFINITY : -bias[j].x;
    }
    const float i0 = L[0] == 0.f ? 0.f : __fdiv_rn(1.f, L[0]);
    const float i1 = L[1] == 0.f ? 0.f : __fdiv_rn(1.f, L[1]);
    const float scale = __fdiv_rn(1.f, unit);
#pragma unroll
    for (int gr = 0; gr < 4; ++gr)
#pragma unroll
      for (int ti = 0; ti < 2; ++ti)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          // O_1 from D; rounded alone, so that equal branches with lambda = 1 give exactly 0
          o[gr][ti][i] = __fmul_rn(__fmul_rn(fmaf(c, o[gr][ti][i + 1], o[gr][ti][i]), i0), scale);
          o[gr][ti][i + 1] = __fmul_rn(__fmul_rn(o[gr][ti][i + 1], i1), scale);
        }
    if constexpr (TL::PER_HEAD > 1) {
      // the head's other warps hand their states to its first
      constexpr int OTHERS = TL::PER_HEAD - 1;
      float* sm_o = reinterpret_cast<float*>(smem + STAGES * TL::STAGE_BYTES);  // [HB][OTHERS][ROWS][W]
      float* sm_ml = sm_o + OTHERS * HB * ROWS * W;                            // [HB][OTHERS][ROWS][2]
      bar_consumers<CW * 32>();  // the entry before has been joined
      if (part) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = (hb * OTHERS + part - 1) * ROWS + 2 * tq + j;
          if (gq == 0) *reinterpret_cast<float2*>(sm_ml + 2 * row) = make_float2(M[j], L[j]);
#pragma unroll
          for (int gr = 0; gr < 4; ++gr)
            *reinterpret_cast<float4*>(sm_o + row * W + gr * 32 + gq * 4) =
                make_float4(o[gr][0][j], o[gr][0][2 + j], o[gr][1][j], o[gr][1][2 + j]);
        }
      }
      bar_consumers<CW * 32>();
      if (part == 0) {
#pragma unroll 1
        for (int w = 0; w < OTHERS; ++w)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int row = (hb * OTHERS + w) * ROWS + 2 * tq + j;
            const float2 other = *reinterpret_cast<const float2*>(sm_ml + 2 * row);
            // a state without keys, or with none above -inf, has M = -inf and nothing to add;
            // only a NaN among its sums is passed on
            const float top = fmaxf(M[j], other.x);
            float f0 = __fmul_rn(L[j], M[j] == -INFINITY ? 1.f : ex2(M[j] - top));
            float f1 = __fmul_rn(other.y, other.x == -INFINITY ? 1.f : ex2(other.x - top));
            M[j] = top;
            L[j] = f0 + f1;
            const float inv = L[j] == 0.f ? 0.f : __fdiv_rn(1.f, L[j]);
            f0 = __fmul_rn(f0, inv);
            f1 = __fmul_rn(f1, inv);
#pragma unroll
            for (int gr = 0; gr < 4; ++gr) {
              const float4 v = *reinterpret_cast<const float4*>(sm_o + row * W + gr * 32 + gq * 4);
              o[gr][0][j] = fmaf(o[gr][0][j], f0, v.x * f1);
              o[gr][0][2 + j] = fmaf(o[gr][0][2 + j], f0, v.y * f1);
              o[gr][1][j] = fmaf(o[gr][1][j], f0, v.z * f1);
              o[gr][1][2 + j] = fmaf(o[gr][1][2 + j], f0, v.w * f1);
            }
          }
      }
    }
    if (part == 0) {
      const bool whole = entry_begin >= range_begin && entry_end <= range_end;
      if (whole) {
        // a unit's 128 channels lie in the 8 lanes of a column pair, 16 to each
        float y[4][4], ss = 0.f;
#pragma unroll
        for (int gr = 0; gr < 4; ++gr)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[gr][i] = fmaf(-lam, o[gr][i >> 1][2 * (i & 1) + 1], o[gr][i >> 1][2 * (i & 1)]);
            ss = fmaf(y[gr][i], y[gr][i], ss);
          }
        float f = 1.f;
        if (a.apply_norm) {
#pragma unroll
          for (int s = 4; s <= 16; s <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
          f = rsqrtf(ss * (1.f / W) + a.eps) * (1.f - __ldg(a.lambda_init));
        }
        const int64_t off = b * a.os[0] + (int64_t)u * a.os[1] + gq * 4;
#pragma unroll
        for (int gr = 0; gr < 4; ++gr)
          if (is_unit && in_bounds(off + gr * 32, 4, a.ext_out, a.cache.dev_status, a.cache.dbg_status))
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + off + gr * 32) =
                make_uint2(pack_bf16(y[gr][0] * f, y[gr][1] * f), pack_bf16(y[gr][2] * f, y[gr][3] * f));
      } else {
        const int slot = entry_begin < range_begin ? 0 : 1;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!is_unit) continue;
          const int64_t rec = (((int64_t)blockIdx.x * 2 + slot) * HB + hb) * ROWS + 2 * tq + j;
          if (in_bounds(rec * W, W, a.ext_ws_o, a.cache.dev_status, a.cache.dbg_status)) {
#pragma unroll
            for (int gr = 0; gr < 4; ++gr)
              *reinterpret_cast<float4*>(a.ws_o + rec * W + gr * 32 + gq * 4) =
                  make_float4(o[gr][0][j], o[gr][0][2 + j], o[gr][1][j], o[gr][1][2 + j]);
          }
          if (gq == 0 && in_bounds(rec * 2, 2, a.ext_ws_ml, a.cache.dev_status, a.cache.dbg_status))
            *reinterpret_cast<float2*>(a.ws_ml + rec * 2) = make_float2(M[j], L[j]);
        }
      }
    }
    at = stop;
    if (at == range_end) break;
    entry_begin = entry_end;
    do ++b;  // the next entry that has keys
    while (kv4_len(a, b) == 0);
  }
}

// The output of one unit (V1 head or V2 pair) from its branches' attention outputs, channel
// `c` of the W threads with `mine`: the difference, and V1's norm and scale; zero for an entry
// without `keys`, whatever lambda and eps are. All threads of the block take part; `red` holds 4
// floats.
__device__ __forceinline__ void store_unit(const DecodeKv4Args& a, int b, int u, int c, bool mine, bool keys, float o1,
                                           float o2, float* red) {
  float y = keys ? o1 - __ldg(a.lambda + u) * o2 : 0.f;
  if (a.apply_norm && keys) {
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

// Joins the states of the units that several blocks share, and writes the zero rows of entries
// without keys: one block per output unit (V1 head or V2 pair) and entry. A state's weight
// 2^(M_s - M) is computed once by one thread; each of SLICES warps then adds every SLICES-th
// state, four channels to a lane and both rows, and their sums are added in order. (103 states
// took 52 us with a thread to a channel walking them all.) SLICES = 16 for few entries with
// many states each, 4 for many with few: 222 states of one entry took 15 us instead of 32,
// 10 states each of 24 entries 18 us instead of 29.
// Few entries also split a unit's channels over W / CH blocks, where no norm runs over them.
template <int SLICES, int CH>
__global__ void __launch_bounds__(32 * SLICES) decode_kv4_combine_kernel(DecodeKv4Args a) {
  constexpr int JOIN = 32 * SLICES;  // states whose weights are held at a time
  constexpr int LANES = CH / 4, AT_ONCE = 32 / LANES;  // lanes of a state, states of a warp at once
  __shared__ float weight[2][JOIN];
  __shared__ float4 part[SLICES * AT_ONCE][2][LANES];
  __shared__ float red[2][SLICES];
  __shared__ uint32_t sums[SLICES];
  constexpr int THREADS = 32 * SLICES;
  const int u = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c0 = blockIdx.z * CH;
  // the unit's head, row and head tile
  const int head = a.v1 ? u : 2 * u / a.group, row = 2 * u - head * a.group;
  const int ck = KEYS * (CW / a.heads), tiles = (a.group + ROWS - 1) / ROWS;
  const int HQ = a.H / a.heads * tiles, tile_h = head / a.heads * tiles + row / ROWS;
  const uint32_t n = (kv4_len(a, b) + ck - 1) / ck;
  uint32_t T, begin;
  if (!a.kv_len) {
    T = a.B * n;
    begin = b * n;
  } else {
    uint32_t all = 0, lower = 0;
    for (int i = tid; i < a.B; i += THREADS) {
      const uint32_t chunks = (kv4_len(a, i) + ck - 1) / ck;
      all += chunks;
      if (i < b) lower += chunks;
    }
    T = block_sum(all, sums, SLICES);
    begin = block_sum(lower, sums, SLICES);
  }
  const Kv4Cuts cuts(T, a.groups);
  const uint32_t i0 = n ? cuts.range_of(begin) : 0, i1 = n ? cuts.range_of(begin + n - 1) : 0;
  cudaGridDependencySynchronize();  // the split kernel's states
  if (n && i0 == i1) return;        // finished there
  // state s: slot 1 of range i0's block, then slot 0 of the ranges after it
  const int splits = n ? (int)(i1 - i0) + 1 : 0;
  const int64_t step = 2LL * HQ * a.heads * ROWS;
  const int64_t rec0 = (((int64_t)i0 * HQ + tile_h) * 2 * a.heads + head % a.heads) * ROWS + row % ROWS;
  auto record = [&](int s) { return rec0 + (s ? s * step : (int64_t)a.heads * ROWS); };
  const bool ok =
      !splits ||
      (in_bounds(record(splits - 1) * 2, 4, a.ext_ws_ml, a.cache.dev_status, a.cache.dbg_status) &&
       in_bounds(record(splits - 1) * W, 2 * W, a.ext_ws_o, a.cache.dev_status, a.cache.dbg_status));
  const int have = ok ? splits : 0;

  // (M, sum) of both rows of state s
  auto state = [&](int s) { return *reinterpret_cast<const float4*>(a.ws_ml + 2 * record(s)); };
  float M[2] = {-INFINITY, -INFINITY};
  for (int s = tid; s < have; s += THREADS) {
    const float4 v = state(s);
    M[0] = fmaxf(M[0], v.x);
    M[1] = fmaxf(M[1], v.z);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    M[e] = warp_max(M[e]);
    if (lane == 0) red[e][warp] = M[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int w = 0; w < SLICES; ++w) M[e] = fmaxf(M[e], red[e][w]);

  float L[2] = {0.f, 0.f};
  float4 O[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s0 = 0; s0 < have; s0 += JOIN) {
    const int held = min(JOIN, have - s0);
    __syncthreads();
    if (tid < held) {
      const float4 v = state(s0 + tid);
      // a state without keys has M = -inf and nothing to add; only a NaN is passed on. kJoin
      // bounds the sum of all weights by 1: a key counts for at most 2^kSlack in a state's L,
      // and an entry has 2^30 keys at most
      const float f0 = __fmul_rn(__fmul_rn(v.y, kJoin), v.x == -INFINITY ? 1.f : ex2(v.x - M[0]));
      const float f1 = __fmul_rn(__fmul_rn(v.w, kJoin), v.z == -INFINITY ? 1.f : ex2(v.z - M[1]));
      weight[0][tid] = f0;
      weight[1][tid] = f1;
      L[0] += f0;
      L[1] += f1;
    }
    __syncthreads();
#pragma unroll 4
    for (int s = warp * AT_ONCE + lane / LANES; s < held; s += SLICES * AT_ONCE) {
      const float4* po = reinterpret_cast<const float4*>(a.ws_o + record(s0 + s) * W + c0) + lane % LANES;
      const float4 v0 = po[0], v1 = po[W / 4];
      const float f0 = weight[0][s], f1 = weight[1][s];
      O[0] = make_float4(fmaf(v0.x, f0, O[0].x), fmaf(v0.y, f0, O[0].y), fmaf(v0.z, f0, O[0].z), fmaf(v0.w, f0, O[0].w));
      O[1] = make_float4(fmaf(v1.x, f1, O[1].x), fmaf(v1.y, f1, O[1].y), fmaf(v1.z, f1, O[1].z), fmaf(v1.w, f1, O[1].w));
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    L[e] = warp_sum(L[e]);
    if (lane == 0) red[e][warp] = L[e];
    part[warp * AT_ONCE + lane / LANES][e][lane % LANES] = O[e];
  }
  __syncthreads();
  const int c = tid % CH;  // the first CH threads finish, a channel each
  float res[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float l = 0.f, o = 0.f;
    for (int w = 0; w < SLICES; ++w) l += red[e][w];
#pragma unroll 8
    for (int w = 0; w < SLICES * AT_ONCE; ++w) o += reinterpret_cast<const float*>(part[w][e])[c];
    res[e] = l == 0.f ? 0.f : o / l;
  }
  __syncthreads();
  store_unit(a, b, u, c0 + c, tid < CH, n != 0, res[0], res[1], red[0]);
}

// Heads of a block: neighbours read together (one run of 144 HB bytes per token) when the
// cache keeps them side by side. On the full-size step copies alone took 430 us with runs of
// 144 bytes, 390 with 288 and 371 with 576 (the cache once at 6.5 TB/s).
static int kv4_heads(int H, int64_t head_stride) {
  if (H > 1 && head_stride != kKv4Record) return 1;
  return H % 4 == 0 ? 4 : (H % 2 == 0 ? 2 : 1);
}

// Groups of blocks (Kv4Cuts): `num_splits` for each entry on average if that is given, else as
// many as run at once, but not so many that the chunks of full-length entries do not give each
// kMin. States are kept for two entries of every block. Entries stay whole up to 4 chunks, or as
// many as an eighth of the blocks that gives, to 20: a chunk takes a block 0.8 us, what sharing
// costs grows with the entries (64 entries x 8 heads of 300 tokens: 13 us whole, 19 shared; 8
// entries 13 and 9; 600 tokens, 64 entries: 22 and 23).
void decode_kv4_plan(DecodeKv4Args* a, int num_splits) {
  constexpr int64_t kMin = 2;
  a->heads = kv4_heads(a->H, a->cache.stride[2]);
  const int64_t ck = KEYS * (CW / a->heads), per_entry = (a->cache.L + ck - 1) / ck;
  const int64_t HQ = a->H / a->heads * ((a->group + ROWS - 1) / ROWS);
  a->chunks = (int64_t)a->B * per_entry;
  int64_t groups = num_splits ? (int64_t)num_splits * a->B : 148 * kBlocksPerSm / HQ;
  const int64_t most = num_splits ? a->chunks : (a->chunks + kMin - 1) / kMin;
  if (groups > most) groups = most;
  if (groups > (1 << 16)) groups = 1 << 16;
  const int64_t eighth = a->B * HQ / 8, whole = eighth < 4 ? 4 : (eighth < 20 ? eighth : 20);
  a->by_entry = !num_splits && per_entry <= whole;
  if (a->by_entry) groups = a->B;
  a->groups = groups < 1 ? 1 : (int)groups;
  a->blocks = a->groups * HQ;
  a->states = a->by_entry ? 0 : a->blocks * 2 * a->heads * ROWS;
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

template <int HB>
static cudaError_t launch_split(const DecodeKv4Args& a, cudaStream_t stream) {
  using TL = Tile<HB>;
  const bool paged = a.cache.block_table != nullptr;
  const int page = 1 << a.cache.page_shift;
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  Kv4Load how = kRows;
  if (!paged && kv4_map<HB>(&map, a.cache, a.H, a.cache.L, a.B, TL::CK)) how = kTma;
  if (paged && page >= 8 &&
      kv4_map<HB>(&map, a.cache, a.H, page, a.cache.num_pages, page < TL::CK ? page : TL::CK))
    how = kTmaPaged;
  void (*const fns[3])(CUtensorMap, DecodeKv4Args) = {decode_kv4_split_kernel<HB, kTma>,
                                                      decode_kv4_split_kernel<HB, kTmaPaged>,
                                                      decode_kv4_split_kernel<HB, kRows>};
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
  const cudaError_t e =
      a.heads == 4 ? launch_split<4>(a, stream) : (a.heads == 2 ? launch_split<2>(a, stream) : launch_split<1>(a, stream));
  if (e != cudaSuccess || a.by_entry) return e;
  // launched while the last blocks still run; the kernel waits for them itself. (With the split
  // kernel launched early too, behind the join of the call before, ragged batches took 45 us
  // instead of 39: its blocks then hold the SMs that the join needs.)
  const bool many = a.groups > 64 * (int64_t)a.B, spread = many && !a.apply_norm;
  return kv4_launch_early(spread ? decode_kv4_combine_kernel<16, 32>
                                 : (many ? decode_kv4_combine_kernel<16, W> : decode_kv4_combine_kernel<4, W>),
                          dim3(a.H * a.group / 2, a.B, spread ? W / 32 : 1), dim3(many ? 512 : 128), 0, stream, a);
}

}  // namespace diffattn
