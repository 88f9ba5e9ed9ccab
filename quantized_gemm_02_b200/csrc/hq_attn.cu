// Attention of one new token per sequence over the paged key-value cache.
//
// The operation reads each cached key and value once and does 4 G D flops per
// token and kv head with them (G query heads share a kv head): 1 to 16 flops
// a byte, far under what the tensor cores need, so HBM bounds it and the
// kernel is built around the stream of cache units (16 tokens of one head,
// contiguous, see hq_cache.cu):
//
//   * The units of all sequences and kv heads form one line, cut into equal
//     parts for the SMs and, inside an SM, for its warps; ragged lengths
//     therefore balance to one unit, and lengths are read on the device (a
//     captured call serves growing sequences).  A warp consumes its units
//     from a private ring that producer warps fill with one bulk copy a step;
//     warps meet only at the end.
//   * Tokens are the M side of m16n8k16 MMAs and the query heads the N side:
//     S^T = K Q^T, O^T = V^T P^T.  Eight heads fill N, no row of the MMA is
//     padding, and every cache byte is read by exactly one lane, so the cache
//     is stored in fragment order and converted in registers on the way (no
//     transposition, no second pass through shared memory).  The tcgen05 path
//     would need the converted tile written back to shared or tensor memory,
//     and 128 tokens per tile, for an MMA that is idle anyway.
//   * Softmax in base 2 with a running reference per head; the reference only
//     moves when a score exceeds it by 2^LIM, so most units need no exchange
//     between lanes.
//   * Parts of an item (a sequence's kv head) are joined by their log sums:
//     warps of a CTA through shared memory, CTAs through the workspace by the
//     last one to arrive, always in the order of the tokens.
//
// Measured, of the floor of one read of the attended cache at 6.55 TB/s:
// 64 x 8192 tokens x 8 heads x 128, E4M3 (1.09 GB) 170 us under a profiler,
// 98%; bf16 ragged to 8192 97% (three warps with 256 channels: 90%); 8 x
// ~107000 tokens, NVFP4 (1.01 GB) 206 us, 75%.  There, issue slots are 0.61
// used and the ALU pipe 61%, with four warps a scheduler of which 1.4 are
// ready: too few for the chains of conversions and MMAs of a unit (324
// instructions), and SMs idle 9% of the time at the ends.  Ragged batches of
// 0.3 GB 47 to 67 us of floor in 62 to 81 us, 51 to 78%: some 5 us to the first
// unit, 5 to 8 to join, and SMs that end up to 15% apart.  One sequence of 4097
// tokens: 14.3 us, latency (each round trip through L2 in the join is 1 to
// 2 us).
//
// Arithmetic.  Scores and sums are fp32.  bf16 caches multiply in bf16 with
// each weight split into three bf16 numbers, together its 24 bits (two, 2^-17
// of it, were 0 to 1% faster, 3% with 16 heads of 256 channels).  E4M3 and
// NVFP4 codes (and code times block scale) are exact in fp16, so those caches
// multiply in fp16, with q scaled by a power of two per head into fp16's range
// (exact down to 2^-39 of the head's largest) and weights rounded to fp16
// around a reference of 2^10.  That is 2^-11 of a weight, under a hundredth of
// the step of what is held (two fp16 numbers, 2^-22: E4M3 64 ragged x 8192
// 64.8 -> 65.8 us, 33 ragged x 16384 with wide heads 82.6 -> 87.2, NVFP4 8 x
// 107000 229 -> 250, and bf16 results 0.0001 to 0.0002 of their norm from those
// of fp32 weights instead of 0.0007 to 0.0008, where their own rounding is
// 0.0017).  E4M3 values carry an fp32 scale per token: it multiplies the weight,
// and those products have a reference of their own, so that any range of scales
// keeps the weight's precision.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "hq_internal.cuh"

namespace hq {

struct AttnArgs {
  KvArgs kv;
  int num_pages;
  int B, q_heads, group;       // query heads per kv head
  int hgroups;                 // groups of GT query heads per kv head
  const uint16_t *q;
  long long qs;                // stride between sequences, elements
  const int32_t *page_table;
  int max_pages;
  const int32_t *lengths;
  float scale;                 // softmax scale * log2(e)
  int window;
  uint16_t *out;
  long long os;
  float *lse;
  int *counters;               // [CTAs]
  float *parts;                // [CTAs][2] partial records
};

// The tokens a sequence's query sees: [first, len).
__device__ __forceinline__ int attn_range(const AttnArgs &a, int b, int &first) {
  int n = a.lengths[b];
  const int most = a.max_pages * a.kv.page;  // at most 2^30
  if (n < 0 || n > most) {
    set_device_error(HQ_ERR_DEVICE_INDEX);
    n = n < 0 ? 0 : most;
  }
  first = a.window > 0 && n > a.window ? n - a.window : 0;
  return n;
}
// Steps of TOK tokens, aligned to multiples of TOK in the sequence.
template <int TOK>
__device__ __forceinline__ int attn_steps(const AttnArgs &a, int b) {
  int first;
  const int n = attn_range(a, b, first);
  return n ? (int)(((long long)n + TOK - 1) / TOK) - first / TOK : 0;
}

// ---- fragments ---------------------------------------------------------------
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 8 x 8 transposition of 16-bit values held as MMA fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool BF>  // the first of a chain: c = A B
__device__ __forceinline__ void mma16816_new(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// ---- shape of a kernel ---------------------------------------------------------
// NT = 8-head tiles per item.  W consumer warps, each with a ring of STAGES
// units, and P producer warps (a lane's copies are issued one after the
// other, some 150 cycles each: one producer held NVFP4 caches at 60% of HBM).  A partial record is GT x D normalised outputs
// and GT log2 sums; a warp leaves at most two: one in its drained ring, the
// other, written while the ring is in use, beside the rings or, where records
// are large, in the workspace (so in L2).
constexpr int ATTN_SMEM = 227 * 1024 - 1024;  // what a CTA may have, less the static part
constexpr int ATTN_HEAD = 9728;               // barriers and bookkeeping
constexpr int ATTN_MAX_CTAS = 256;
template <int FMT, int D, int NT>
struct AttnShape {
  static constexpr int GT = 8 * NT;
  static constexpr int UNIT = kv_unit_bytes(FMT, D);
  // A step is one unit, or two of the small ones: half the handshakes and
  // copies, and two independent chains of MMAs.
  static constexpr int STEP = FMT == A_NVFP4 || UNIT <= 2304 ? 2 : 1, TOK = 16 * STEP, BYTES = STEP * UNIT;
  static constexpr int PART = GT * (D + 4) * 4;  // bytes; the sums padded to 16 per head
  static constexpr bool FAR = GT * D >= 2048;    // first records in the workspace
  static constexpr int fit(int w) { return ((ATTN_SMEM - ATTN_HEAD) / w - (FAR ? 0 : PART)) / BYTES; }
  // W + P warps are a multiple of four, one per scheduler: 16 warps may have
  // 128 registers a lane, 12 168 and 8 or 4 255.  Of the counts that the
  // registers allow (6 per output tile and 16 channels, and some 70 more), the
  // largest that keeps 120 KB on its way.
  static constexpr int REGS = NT * (D / 16) * 6;
  static constexpr bool deep(int w) { return fit(w) >= 2 && w * fit(w) * BYTES >= 120 * 1024; }
  static constexpr int W = REGS <= 48 && deep(14) ? 14 : REGS <= 96 && deep(10) ? 10 : deep(7) ? 7 : 3;
  static constexpr int P = W >= 10 ? 2 : 1;
  static constexpr int STAGES = fit(W) < 12 ? fit(W) : 12;
  static constexpr int SMEM = ATTN_HEAD + W * ((FAR ? 0 : PART) + STAGES * BYTES);
  static constexpr size_t workspace(int sms) {  // after the counters
    return (size_t)sms * PART * (2 + (FAR ? W : 0));
  }
  static_assert(STAGES >= 2 && STAGES * BYTES >= PART, "ring too small");
};
constexpr int ATTN_RINGS = 15 * 12;  // most (warp, stage) pairs

struct AttnUnit {        // what the producer says of a step
  int b, it, u, nu;      // sequence, head group, the step's place in its item and the item's steps
};
struct AttnSeg {         // a part of an item that a warp leaves behind
  int start;             // the item's first step in the line
  int b, it, nu;
  int flags;             // 1: present, 2: holds the item's first step, 4: its last
};

struct AttnRun {         // segments of one item
  unsigned members;
  int first, begins, ends;
};

struct AttnHead {
  uint64_t full[ATTN_RINGS], empty[ATTN_RINGS];
  union {
    struct {                   // while units are streamed
      AttnUnit unit[ATTN_RINGS];
      int before[512];         // steps of the sequences before a thread's share
    };
    struct {                   // then, of the join
      float weight[16 * 32], run_lse[16 * 32];
    };
  };
  AttnRun run[30];
  int meta[ATTN_RINGS];        // valid tokens [lo, hi) in bits 0..5 and 6..11, and flags:
  AttnSeg seg[30];             // [W][2]
};
enum { ATTN_LAST = 1 << 12, ATTN_BAD = 1 << 13 };  // the item's last step; unit k's page does not exist (BAD << k)
// A walk along the line of steps.
template <int TOK>
struct AttnWalk {
  int b, it, u, nu, u0, len, first;
  __device__ __forceinline__ void open(const AttnArgs &a) {
    len = attn_range(a, b, first);
    u0 = first / TOK;
    nu = len ? (int)(((long long)len + TOK - 1) / TOK) - u0 : 0;
  }
  // to the next unit; there is one.  True if it is another item's.
  __device__ __forceinline__ bool next(const AttnArgs &a, int items) {
    if (++u < nu) return false;
    u = 0;
    if (++it < items) return true;
    it = 0;
    do {
      ++b;
      open(a);
    } while (nu == 0 && b < a.B - 1);
    return true;
  }
};

// n things in `parts` consecutive parts that differ by one at most.
struct AttnSplit {
  int each, more;  // the first `more` parts have one more
  __device__ __forceinline__ int begin(int part) const { return part * each + min(part, more); }
  __device__ __forceinline__ int part_of(int i) const {
    const int n = more * (each + 1);
    return i < n ? i / (each + 1) : more + (i - n) / each;
  }
};

__device__ __forceinline__ int atom_add_acq_rel(int *p, int v) {
  int r;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
  return r;
}
__device__ __forceinline__ unsigned upto_mask(int lane) { return (2u << lane) - 1u; }
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {  // does not suspend the warp
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(AttnShape<FMT, D, NT>::W * 32 + AttnShape<FMT, D, NT>::P * 32, 1) attn_kernel(AttnArgs a) {
  using S = AttnShape<FMT, D, NT>;
  constexpr int W = S::W, P = S::P, STAGES = S::STAGES, UNIT = S::UNIT, GT = S::GT, PART = S::PART;
  constexpr int STEP = S::STEP, TOK = S::TOK, BYTES = S::BYTES;
  constexpr int CB = kv_code_bytes(FMT, D), SB = kv_scale_bytes(FMT, D);
  constexpr int THREADS = (W + P) * 32;
  constexpr bool BF = FMT == A_BF16;
  constexpr float LIM = BF ? 8.f : 15.f, SHIFT = BF ? 0.f : 10.f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned s_scan[W + P];
  __shared__ int s_last[2], s_from[6];
  __shared__ volatile int s_stop;
  AttnHead *head = reinterpret_cast<AttnHead *>(smem);
  static_assert(sizeof(AttnHead) <= ATTN_HEAD && W * STAGES <= ATTN_RINGS, "bookkeeping");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int items = a.kv.H * a.hgroups;
  auto near_record = [&](int w) {  // a warp's part of an item begun before
    return S::FAR ? a.parts + ((size_t)gridDim.x * 2 + (size_t)blockIdx.x * W + w) * (PART / 4)
                  : reinterpret_cast<float *>(smem + ATTN_HEAD + W * STAGES * BYTES) + w * (PART / 4);
  };

  if (tid < W * STAGES) {
    mbar_init(&head->full[tid], 1);
    mbar_init(&head->empty[tid], 1);
    fence_barrier_init();
  }
  if (tid < 2 * W) head->seg[tid].flags = 0;
  if (tid == 0) s_stop = 0;

  // The line's length: each thread counts the units of its share of the
  // sequences.  Empty sequences get their zeros from one of the CTAs.
  const int per = (a.B + THREADS - 1) / THREADS;
  unsigned mine = 0;
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    const int n = b < a.B ? attn_steps<TOK>(a, b) : 1;
    // (32 bits hold the line, or the call is refused below; a share stops short of wrapping around)
    if (b < a.B) mine = min(mine + (unsigned)n, 1u << 30);
    unsigned empty = __ballot_sync(0xffffffffu, n == 0 && b % gridDim.x == blockIdx.x);
    while (empty) {
      const int eb = __shfl_sync(0xffffffffu, b, __ffs(empty) - 1);
      empty &= empty - 1;
      for (int i = lane; i < a.q_heads * (D / 8); i += 32)
        *reinterpret_cast<uint4 *>(a.out + eb * a.os + (size_t)i * 8) = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int i = lane; i < a.q_heads; i += 32) a.lse[(size_t)eb * a.q_heads + i] = -INFINITY;
    }
  }
  unsigned incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl = min(incl + v, 1u << 30);
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  const int shares = (a.B + per - 1) / per;
  unsigned long long before = incl - mine, sum = 0;
  for (int w = 0; w * 32 < shares; ++w) {
    if (w < warp) before += s_scan[w];
    sum += s_scan[w];
  }
  head->before[tid] = (int)before;
  if (sum * items >= 1ull << 30) {  // steps are counted in 32 bits
    if (tid == 0) set_device_error(HQ_ERR_UNSUPPORTED);
    return;
  }
  const int total = (int)sum * items;
  // A step per warp at least.  Where some warps would have two (or three, four)
  // and others one less, all have the larger number and fewer CTAs take part:
  // the same time for the steps, fewer records to join (1 x 4097 tokens, bf16:
  // 13.8 us instead of 15.1).
  const int most = max((total + W * (int)gridDim.x - 1) / (W * (int)gridDim.x), 1);
  const int ctas = most <= 4 ? (total + most * W - 1) / (most * W) : (int)gridDim.x;
  if (total == 0 || (int)blockIdx.x >= ctas) return;
  const int each = total / ctas;
  const AttnSplit line{each, total - each * ctas};
  const int c_begin = line.begin(blockIdx.x), c_steps = line.begin(blockIdx.x + 1) - c_begin;
  // this warp's steps (producer p: lane i has warp i P + p's)
  const int wi = warp < W ? warp : min(lane * P + warp - W, W);
  const AttnSplit mine_of{c_steps / W, c_steps % W};
  const int w_begin = c_begin + mine_of.begin(wi);
  int left = wi < W ? mine_of.each + (wi < mine_of.more) : 0;
  __syncthreads();
  AttnWalk<TOK> pw{};  // where they begin
  if (left > 0) {
    const int seq = w_begin / items;
    int lo = 0;  // the last share that begins at or before it
    for (int o = shares > 1 ? 1 << (31 - __clz(shares - 1)) : 0; o > 0; o >>= 1)
      if (lo + o < shares && head->before[lo + o] <= seq) lo += o;
    int off = w_begin - head->before[lo] * items;
    for (pw.b = lo * per;; ++pw.b) {
      pw.open(a);
      if (off < pw.nu * items || pw.b >= a.B - 1) break;
      off -= pw.nu * items;
    }
    // (kept in range even if someone changes the lengths meanwhile)
    const int nu = max(pw.nu, 1);
    pw.it = min(off / nu, items - 1);
    pw.u = min(off - pw.it * nu, nu - 1);
  }

  if (warp >= W) {
    // A producer: each lane walks one consumer warp's part of the line.
    int to_issue = left, issued = 0, stage = 0, pidx = 0, psub = 0, pg[STEP] = {};
    uint32_t parity = 1;
    const int upp = a.kv.page_units;
    const int32_t *pages = a.page_table;
    // The pages of the step's units.  Entries before the window are not used,
    // those past the length not read; the second unit may be on the next page.
    auto fetch = [&](bool turned) {
      if (turned) {
        pages = a.page_table + (size_t)pw.b * a.max_pages;
        pidx = (pw.u0 + pw.u) * STEP / upp;
        psub = (pw.u0 + pw.u) * STEP - pidx * upp;
      } else {
        psub += STEP;
        if (psub < upp) {
          if (STEP == 1 || psub + 1 < upp) {
            if (STEP == 2) pg[1] = pg[0];
            return;
          }
        } else {
          psub -= upp;
          ++pidx;
          if (STEP == 2 && psub >= upp) {  // pages of one unit
            psub -= upp;
            ++pidx;
          }
        }
      }
      const int at = (pw.u0 + pw.u) * TOK;
      pg[0] = pages[pidx];  // (also where the window begins in the second unit: later steps are on this page)
      if constexpr (STEP == 2) pg[1] = at + 16 >= pw.len ? -1 : psub + 1 < upp ? pages[pidx] : pages[pidx + 1];
    };
    if (to_issue > 0) fetch(true);
    unsigned long long idle = 0;
    while (__any_sync(0xffffffffu, to_issue > 0)) {
      const int slot = wi * STAGES + stage;
      const bool ready = to_issue > 0 && (issued < STAGES || mbar_test(&head->empty[slot], parity));
      if (ready) {
        const int tok0 = (pw.u0 + pw.u) * TOK, lo = max(pw.first - tok0, 0), hi = min(pw.len - tok0, TOK);
        int meta = lo | hi << 6 | (pw.u + 1 == pw.nu ? ATTN_LAST : 0), bytes = 0;
        bool go[STEP];
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
          const bool used = lo < 16 * k + 16 && hi > 16 * k;
          go[k] = used && pg[k] >= 0 && pg[k] < a.num_pages;
          if (used && !go[k]) {
            meta |= ATTN_BAD << k;
            set_device_error(HQ_ERR_DEVICE_INDEX);
          }
          if (go[k]) bytes += UNIT;
        }
        head->unit[slot] = AttnUnit{pw.b, pw.it, pw.u, pw.nu};
        head->meta[slot] = meta;
        const size_t head_off = (size_t)(pw.it / a.hgroups) * upp;
        uint8_t *dst = smem + ATTN_HEAD + slot * BYTES;
        const uint8_t *src = a.kv.pages + (size_t)pg[0] * a.kv.page_bytes + (head_off + psub) * UNIT;
        if (bytes) mbar_arrive_expect_tx(&head->full[slot], bytes);
        else mbar_arrive(&head->full[slot]);
        if constexpr (STEP == 1) {
          if (bytes) bulk_g2s(dst, src, UNIT, &head->full[slot]);
        } else if (bytes == BYTES && psub + 1 < upp) {
          bulk_g2s(dst, src, BYTES, &head->full[slot]);
        } else {
          const int sub = psub + 1 < upp ? psub + 1 : 0;
          if (go[0]) bulk_g2s(dst, src, UNIT, &head->full[slot]);
          if (go[1]) bulk_g2s(dst + UNIT, a.kv.pages + (size_t)pg[1] * a.kv.page_bytes + (head_off + sub) * UNIT, UNIT, &head->full[slot]);
        }
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          parity ^= 1u;
        }
        if (--to_issue > 0) {
          fetch(pw.next(a, items));
        }
      }
      if (__any_sync(0xffffffffu, ready)) {
        idle = 0;
      } else {
        __nanosleep(32);
        const unsigned long long now = __shfl_sync(0xffffffffu, global_timer_ns(), 0);
        if (idle == 0) idle = now;
        const bool late = now - idle > WAIT_LIMIT_NS;
        if (late) set_device_error(HQ_ERR_TIMEOUT);
        if (__any_sync(0xffffffffu, late || s_stop)) break;
      }
    }
  }
  if (warp < W && left > 0) {
    int pos = w_begin;  // the next step, along the line
    uint8_t *ring = smem + ATTN_HEAD + warp * (STAGES * BYTES);
    float *rec0 = near_record(warp);
    AttnUnit cu{pw.b, pw.it, pw.u, pw.nu};  // the item at hand
    int item_start = pos - pw.u;
    uint32_t qf[NT][D / 16][2];  // B fragments of q: k = this lane's channels, n = head g
    float qc[NT][2];             // score multiplier of heads 2t, 2t + 1
    float o[NT][D / 16][4], l[NT][2], ref[NT][2], refv[NT][2];
    bool fresh = true;
    int stage = 0;
    uint32_t parity = 0;

    while (left > 0) {
      const int slot = warp * STAGES + stage;
      auto arrived = [&]() { return __all_sync(0xffffffffu, mbar_wait(&head->full[slot], parity)); };
      if (fresh) {  // the first item is known before its unit is here
        fresh = false;
        if (pos != w_begin && arrived()) {
          cu = head->unit[slot];
          item_start = pos - cu.u;
        }
        const int h = cu.it / a.hgroups, hg = cu.it % a.hgroups;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int hq = hg * GT + nt * 8 + g;
          const bool on = hq < a.group;
          const uint16_t *src = a.q + cu.b * a.qs + (size_t)(h * a.group + (on ? hq : 0)) * D + 8 * t;
          uint4 v[D / 32];
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            v[i] = on ? *reinterpret_cast<const uint4 *>(src + 32 * i) : make_uint4(0, 0, 0, 0);
            if constexpr (!BF) {
              float f[8];
              unpack8(v[i], f);
#pragma unroll
              for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
            }
          }
          float mult = 1.f, sc = a.scale;
          if constexpr (!BF) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int ex = (int)(__float_as_uint(amax) >> 23);
            // the head's largest |q| into [2^13, 2^14)
            const int e = (amax == 0.f || ex == 255) ? 0 : max(ex - 140, -126);
            mult = exp2i(-e);
            sc *= exp2i(e);
            if constexpr (FMT == A_NVFP4) sc *= a.kv.glob[0];
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            if constexpr (BF) {
              qf[nt][2 * i][0] = v[i].x;
              qf[nt][2 * i][1] = v[i].y;
              qf[nt][2 * i + 1][0] = v[i].z;
              qf[nt][2 * i + 1][1] = v[i].w;
            } else {
              float f[8];
              unpack8(v[i], f);
              qf[nt][2 * i][0] = f16x2(f[0] * mult, f[1] * mult);
              qf[nt][2 * i][1] = f16x2(f[2] * mult, f[3] * mult);
              qf[nt][2 * i + 1][0] = f16x2(f[4] * mult, f[5] * mult);
              qf[nt][2 * i + 1][1] = f16x2(f[6] * mult, f[7] * mult);
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            qc[nt][j] = __shfl_sync(0xffffffffu, sc, (2 * t + j) * 4);
            l[nt][j] = 0.f;
            ref[nt][j] = refv[nt][j] = -3e38f;
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
        }
      }

      if (!arrived()) {
        // gave up (recorded): stop the copies, and give those in flight time to land before the CTA goes
        s_stop = 1;
        for (int k = 0; k < STAGES; ++k) {
          mbar_wait(&head->full[warp * STAGES + stage], parity, WAIT_LIMIT_NS / 100);
          if (++stage == STAGES) {
            stage = 0;
            parity ^= 1u;
          }
        }
        break;
      }
      const int meta = head->meta[slot];
      {
        uint8_t *unit = ring + stage * BYTES;
        const int lo = meta & 63, hi = meta >> 6 & 63;  // valid tokens
        const bool edge = lo > 0 || hi < TOK || meta >= ATTN_BAD;
        auto valid = [&](int j) { return j >= lo && j < hi && !(meta & ATTN_BAD << (j >> 4)); };
        if (edge) {
          // what lies past the sequence may be NaN, and 0 * NaN is: zero the values this lane reads
          constexpr int GS = kv_granule(FMT);
#pragma unroll 1
          for (int k = 0; k < STEP; ++k) {
            uint8_t *v = unit + k * UNIT + CB;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              if (valid(16 * k + 2 * t + (i & 1) + 8 * ((i >> 1) & 1))) continue;
              uint8_t *p = v + lane_byte<GS>(lane, i);
              if constexpr (FMT == A_BF16) *reinterpret_cast<uint4 *>(p) = make_uint4(0, 0, 0, 0);
              if constexpr (FMT == A_FP8) *reinterpret_cast<uint2 *>(p) = make_uint2(0, 0);
              if constexpr (FMT == A_NVFP4) *reinterpret_cast<uint32_t *>(p) = 0;
            }
            if constexpr (FMT == A_NVFP4) {
              for (int i = lane; i < D; i += 32)
                if (!valid(16 * k + (i & 15))) v[CB + SB + i] = 0;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }

        // S^T of unit k: rows g and g + 8 (tokens) x heads 2t, 2t + 1.  One unit
        // takes two chains of MMAs, two take one each.
        float acc[NT][2][4];
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
          const uint4 *kv4 = reinterpret_cast<const uint4 *>(unit + k * UNIT) + lane;
          auto qk = [&](int step, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (step < (STEP == 2 ? 1 : 2))
                mma16816_new<BF>(acc[nt][STEP == 2 ? k : step & 1], a0, a1, a2, a3, qf[nt][step][0], qf[nt][step][1]);
              else
                mma16816<BF>(acc[nt][STEP == 2 ? k : step & 1], a0, a1, a2, a3, qf[nt][step][0], qf[nt][step][1]);
            }
          };
          if constexpr (FMT == A_BF16) {
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
              const uint4 v0 = kv4[(2 * b) * 32], v1 = kv4[(2 * b + 1) * 32];
              qk(2 * b, v0.x, v1.x, v0.y, v1.y);
              qk(2 * b + 1, v0.z, v1.z, v0.w, v1.w);
            }
          } else if constexpr (FMT == A_FP8) {
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
              const uint4 v = kv4[b * 32];
              qk(2 * b, e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.z), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.z >> 16));
              qk(2 * b + 1, e4m3x2_to_f16x2(v.y), e4m3x2_to_f16x2(v.w), e4m3x2_to_f16x2(v.y >> 16),
                 e4m3x2_to_f16x2(v.w >> 16));
            }
          } else {
            // this lane's channels 32b + 8t.. lie in 16-channel block 2b + t / 2
            const uint8_t *ksc = unit + k * UNIT + 2 * CB;
            const uint16_t *s0 = reinterpret_cast<const uint16_t *>(ksc + g * (D / 16) + (t >> 1) * (D / 32));
            const uint16_t *s1 = reinterpret_cast<const uint16_t *>(ksc + (g + 8) * (D / 16) + (t >> 1) * (D / 32));
#pragma unroll
            for (int b2 = 0; b2 < D / 64; ++b2) {
              const uint4 v = kv4[b2 * 32];
              const uint32_t p0 = e4m3x2_to_f16x2(s0[b2]), p1 = e4m3x2_to_f16x2(s1[b2]);
              const uint32_t r0 = __byte_perm(p0, 0, 0x1010), r1 = __byte_perm(p1, 0, 0x1010);
              const uint32_t t0 = __byte_perm(p0, 0, 0x3232), t1 = __byte_perm(p1, 0, 0x3232);
              qk(4 * b2, hmul2(e2m1x2_to_f16x2<0>(v.x), r0), hmul2(e2m1x2_to_f16x2<0>(v.y), r1),
                 hmul2(e2m1x2_to_f16x2<1>(v.x), r0), hmul2(e2m1x2_to_f16x2<1>(v.y), r1));
              qk(4 * b2 + 1, hmul2(e2m1x2_to_f16x2<2>(v.x), r0), hmul2(e2m1x2_to_f16x2<2>(v.y), r1),
                 hmul2(e2m1x2_to_f16x2<3>(v.x), r0), hmul2(e2m1x2_to_f16x2<3>(v.y), r1));
              qk(4 * b2 + 2, hmul2(e2m1x2_to_f16x2<0>(v.z), t0), hmul2(e2m1x2_to_f16x2<0>(v.w), t1),
                 hmul2(e2m1x2_to_f16x2<1>(v.z), t0), hmul2(e2m1x2_to_f16x2<1>(v.w), t1));
              qk(4 * b2 + 3, hmul2(e2m1x2_to_f16x2<2>(v.z), t0), hmul2(e2m1x2_to_f16x2<2>(v.w), t1),
                 hmul2(e2m1x2_to_f16x2<3>(v.z), t0), hmul2(e2m1x2_to_f16x2<3>(v.w), t1));
            }
          }
        }

        // Scores above the reference, in base 2.  x: of the weight; y (E4M3):
        // of the weight times the value's scale, which has its own reference.
        float x[NT][STEP][4], y[NT][STEP][4];
        bool raise = false;
        const float *scales = reinterpret_cast<const float *>(unit + 2 * CB);  // E4M3: keys' [16], values' [16]
        auto sum = [&](int nt, int k, int j) { return STEP == 2 ? acc[nt][k][j] : acc[nt][0][j] + acc[nt][1][j]; };
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
          float kscale[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};
          if constexpr (FMT == A_FP8) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              kscale[r] = scales[k * (UNIT / 4) + g + 8 * r];
              lv[r] = lg2(scales[k * (UNIT / 4) + 16 + g + 8 * r]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (FMT == A_FP8) {
                const float sq = sum(nt, k, j) * (qc[nt][j & 1] * kscale[j >> 1]);
                x[nt][k][j] = sq - ref[nt][j & 1];
                y[nt][k][j] = sq + (lv[j >> 1] - refv[nt][j & 1]);
              } else {
                x[nt][k][j] = __fmaf_rn(sum(nt, k, j), qc[nt][j & 1], -ref[nt][j & 1]);
              }
              if (edge && !valid(16 * k + g + 8 * (j >> 1))) x[nt][k][j] = y[nt][k][j] = -INFINITY;
              raise |= x[nt][k][j] > (FMT == A_FP8 ? 64.f : LIM);
              if constexpr (FMT == A_FP8) raise |= y[nt][k][j] > LIM;
            }
        }
        if (__any_sync(0xffffffffu, raise)) {
          // Move the references up to the step's largest score.  The scores are
          // formed again: the first reference, -3e38, has swallowed them.
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float sx[2 * STEP], sy[2 * STEP], mx = -INFINITY, mv = -INFINITY;
#pragma unroll
              for (int i = 0; i < 2 * STEP; ++i) {
                const int k = i >> 1, r = i & 1;
                const bool out = x[nt][k][2 * r + j] == -INFINITY;  // masked
                float q = qc[nt][j], lv = 0.f;
                if constexpr (FMT == A_FP8) {
                  q *= scales[k * (UNIT / 4) + g + 8 * r];
                  lv = lg2(scales[k * (UNIT / 4) + 16 + g + 8 * r]);
                }
                sx[i] = out ? -INFINITY : sum(nt, k, 2 * r + j) * q;
                sy[i] = out ? -INFINITY : sx[i] + lv;
                mx = fmaxf(mx, sx[i]);
                mv = fmaxf(mv, sy[i]);
              }
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
                if constexpr (FMT == A_FP8) mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, k));
              }
              const float r = fmaxf(ref[nt][j], mx - (FMT == A_FP8 ? 0.f : SHIFT));
              float keep = ex2(ref[nt][j] - r);
              ref[nt][j] = r;
              l[nt][j] *= keep;
              if constexpr (FMT == A_FP8) {
                const float rv = fmaxf(refv[nt][j], mv - SHIFT);
                keep = ex2(refv[nt][j] - rv);
                refv[nt][j] = rv;
              }
#pragma unroll
              for (int i = 0; i < 2 * STEP; ++i) {
                x[nt][i >> 1][2 * (i & 1) + j] = sx[i] - ref[nt][j];
                y[nt][i >> 1][2 * (i & 1) + j] = sy[i] - refv[nt][j];
              }
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[nt][i][j] *= keep;
                o[nt][i][2 + j] *= keep;
              }
            }
        }
        constexpr int PARTS = BF ? 3 : 1;  // summands of a weight, each what the ones before lack
        uint32_t pb[NT][STEP][PARTS][2];   // B fragments of P^T: tokens 2t, 2t + 1 (+ 8), head g
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < STEP; ++k) {
            float p[4], w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              p[j] = ex2(x[nt][k][j]);
              w[j] = FMT == A_FP8 ? ex2(y[nt][k][j]) : p[j];
            }
            l[nt][0] += p[0] + p[2];
            l[nt][1] += p[1] + p[3];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float w0 = w[2 * r], w1 = w[2 * r + 1];
#pragma unroll
              for (int i = 0; i < PARTS; ++i) {
                const uint32_t h = BF ? bf16x2(w0, w1) : f16x2(w0, w1);
                pb[nt][k][i][r] = transpose8(h);
                w0 -= bf16_lo(h);
                w1 -= bf16_hi(h);
              }
            }
          }

        // O^T: rows g and g + 8 are channels g (D / 8) + 2i and + 1
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
          const uint4 *vv4 = reinterpret_cast<const uint4 *>(unit + k * UNIT + CB) + lane;
          auto pv = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int j = 0; j < PARTS; ++j) mma16816<BF>(o[nt][i], a0, a1, a2, a3, pb[nt][k][j][0], pb[nt][k][j][1]);
            }
          };
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            if constexpr (FMT == A_BF16) {
              const uint4 v0 = vv4[(4 * q) * 32], v1 = vv4[(4 * q + 1) * 32], v2 = vv4[(4 * q + 2) * 32],
                          v3 = vv4[(4 * q + 3) * 32];
              const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w},
                             w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                pv(4 * q + i, __byte_perm(w0[i], w1[i], 0x5410), __byte_perm(w0[i], w1[i], 0x7632),
                   __byte_perm(w2[i], w3[i], 0x5410), __byte_perm(w2[i], w3[i], 0x7632));
            } else if constexpr (FMT == A_FP8) {
              const uint4 v0 = vv4[(2 * q) * 32], v1 = vv4[(2 * q + 1) * 32];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t a = __byte_perm(i < 2 ? v0.x : v0.y, i < 2 ? v0.z : v0.w, (i & 1) ? 0x7362 : 0x5140);
                const uint32_t c = __byte_perm(i < 2 ? v1.x : v1.y, i < 2 ? v1.z : v1.w, (i & 1) ? 0x7362 : 0x5140);
                pv(4 * q + i, e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(c), e4m3x2_to_f16x2(c >> 16));
              }
            } else {
              const uint4 v = vv4[q * 32];
              const int blk = (g * (D / 64) + q) >> 1;
              const uint16_t *vs = reinterpret_cast<const uint16_t *>(unit + k * UNIT + 2 * CB + SB + blk * 16);
              const uint32_t s01 = e4m3x2_to_f16x2(vs[t]), s23 = e4m3x2_to_f16x2(vs[t + 4]);
              const uint32_t m = 0x0f0f0f0fu;
              const uint32_t e0 = (v.x & m) | ((v.y & m) << 4), e1 = ((v.x >> 4) & m) | (v.y & ~m);
              const uint32_t e2 = (v.z & m) | ((v.w & m) << 4), e3 = ((v.z >> 4) & m) | (v.w & ~m);
              pv(4 * q, hmul2(e2m1x2_to_f16x2<0>(e0), s01), hmul2(e2m1x2_to_f16x2<0>(e1), s01),
                 hmul2(e2m1x2_to_f16x2<0>(e2), s23), hmul2(e2m1x2_to_f16x2<0>(e3), s23));
              pv(4 * q + 1, hmul2(e2m1x2_to_f16x2<1>(e0), s01), hmul2(e2m1x2_to_f16x2<1>(e1), s01),
                 hmul2(e2m1x2_to_f16x2<1>(e2), s23), hmul2(e2m1x2_to_f16x2<1>(e3), s23));
              pv(4 * q + 2, hmul2(e2m1x2_to_f16x2<2>(e0), s01), hmul2(e2m1x2_to_f16x2<2>(e1), s01),
                 hmul2(e2m1x2_to_f16x2<2>(e2), s23), hmul2(e2m1x2_to_f16x2<2>(e3), s23));
              pv(4 * q + 3, hmul2(e2m1x2_to_f16x2<3>(e0), s01), hmul2(e2m1x2_to_f16x2<3>(e1), s01),
                 hmul2(e2m1x2_to_f16x2<3>(e2), s23), hmul2(e2m1x2_to_f16x2<3>(e3), s23));
            }
          }
        }
      }

      __syncwarp();
      if (lane == 0) mbar_arrive(&head->empty[slot]);
      if (++stage == STAGES) {
        stage = 0;
        parity ^= 1u;
      }
      --left;
      ++pos;

      if ((meta & ATTN_LAST) || left == 0) {  // the item, or this warp's part of it, is done
        const bool begins = item_start >= w_begin, ends = meta & ATTN_LAST;
        const int h = cu.it / a.hgroups, hg = cu.it % a.hgroups;
        float *rec = begins ? reinterpret_cast<float *>(ring) : rec0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float s = l[nt][j];
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
            float f1 = s == 0.f ? 0.f : 1.f / s, f2 = 1.f;  // s is 0 where every page was missing
            if constexpr (FMT == A_NVFP4) f1 *= a.kv.glob[1];
            if constexpr (FMT == A_FP8) {
              const float e = refv[nt][j] - ref[nt][j];  // in halves: the scales may span fp32
              f1 *= ex2(0.5f * e);
              f2 = ex2(0.5f * e);
            }
            const float lse2 = s == 0.f ? -INFINITY : ref[nt][j] + lg2(s);
            const int hl = nt * 8 + 2 * t + j, hq = hg * GT + hl;
            if (begins && ends) {
              if (hq < a.group) {
                const size_t row = (size_t)h * a.group + hq;
                uint4 *dst = reinterpret_cast<uint4 *>(a.out + cu.b * a.os + row * D + g * (D / 8));
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = bf16x2(o[nt][4 * i + k][j] * f1 * f2, o[nt][4 * i + k][2 + j] * f1 * f2);
                  dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (a.lse && g == 0) a.lse[(size_t)cu.b * a.q_heads + row] = lse2 * 0.6931471805599453f;
              }
            } else {
              float4 *dst = reinterpret_cast<float4 *>(rec + hl * D + g * (D / 8));
#pragma unroll
              for (int i = 0; i < D / 32; ++i)
                dst[i] = make_float4(o[nt][2 * i][j] * f1 * f2, o[nt][2 * i][2 + j] * f1 * f2,
                                     o[nt][2 * i + 1][j] * f1 * f2, o[nt][2 * i + 1][2 + j] * f1 * f2);
              if (g == 0) rec[GT * D + hl * 4] = lse2;
            }
          }
        if (!(begins && ends) && lane == 0)
          head->seg[2 * warp + (begins ? 1 : 0)] =
              AttnSeg{item_start, cu.b, cu.it, cu.nu, 1 | (begins ? 2 : 0) | (ends ? 4 : 0)};
        fresh = true;
      }
    }
  }
  __syncthreads();

  // Join the parts that the CTA's warps left.  Lane e of every warp has segment
  // e in the order of the tokens; a run of segments up to the next that begins
  // an item is one item's.
  const int fl = lane < 2 * W ? head->seg[lane].flags : 0;
  const unsigned present = __ballot_sync(0xffffffffu, fl & 1), begin = __ballot_sync(0xffffffffu, fl & 2),
                 end = __ballot_sync(0xffffffffu, fl & 4), starts = begin | 1u;
  auto record = [&](int e) {
    return e & 1 ? reinterpret_cast<const float *>(smem + ATTN_HEAD + (e >> 1) * (STAGES * BYTES)) : near_record(e >> 1);
  };
  auto finish = [&](const AttnSeg &sg, int hl, int d, float4 v, float lse2) {  // 4 channels of one head
    const int hq = (sg.it % a.hgroups) * GT + hl;
    if (hq >= a.group) return;
    const size_t row = (size_t)(sg.it / a.hgroups) * a.group + hq;
    *reinterpret_cast<uint2 *>(a.out + sg.b * a.os + row * D + d) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
    if (a.lse && d == 0) a.lse[(size_t)sg.b * a.q_heads + row] = lse2 * 0.6931471805599453f;
  };
  // each segment's weight and each run's log2 sum, by scans within the runs
  int runs;
  {
    const unsigned upto = (2u << lane) - 1u, after = starts & ~upto;
    const int run = 31 - __clz(starts & upto), run_end = after ? __ffs(after) - 2 : 31;
    const unsigned members = present & upto_mask(run_end) & ~((1u << run) - 1u);
    const unsigned heads = __ballot_sync(0xffffffffu, lane == run && members);
    runs = __popc(heads);
    if (warp == 0 && (heads >> lane & 1u))
      head->run[__popc(heads & (upto >> 1))] = AttnRun{members, __ffs(members) - 1, (int)(begin >> lane & 1u), (end & members) != 0};
    for (int hl = warp; hl < GT; hl += W + P) {
      const float ls = fl & 1 ? record(lane)[GT * D + hl * 4] : -INFINITY;
      float m = ls;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, m, o);
        if (lane - o >= run) m = fmaxf(m, u);
      }
      m = __shfl_sync(0xffffffffu, m, run_end);
      const float r = m == -INFINITY ? 0.f : m, w = ex2(ls - r);
      float s = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane - o >= run) s += u;
      }
      s = __shfl_sync(0xffffffffu, s, run_end);
      head->weight[hl * 32 + lane] = s == 0.f ? 0.f : __fdividef(w, s);
      if (lane == run) head->run_lse[hl * 32 + lane] = s == 0.f ? -INFINITY : r + lg2(s);
    }
  }
  __syncthreads();
  // All runs at once, 4 channels of a head at a time.  What spans CTAs goes to
  // the workspace: record [0] of an item begun before this CTA (the first run),
  // [1] of one that goes on after it (the last).
  constexpr int QUADS = GT * D / 4;
  // Each thread has the first two records of FOUR quads on their way at a time.
  constexpr int FOUR = 4;
  for (int i0 = tid; i0 < runs * QUADS; i0 += FOUR * THREADS) {
    float4 p[FOUR][2];
    float w[FOUR][2];
#pragma unroll
    for (int u = 0; u < FOUR; ++u) {
      const int i = i0 + u * THREADS, rn = i / QUADS, x = i - rn * QUADS, hl = x / (D / 4), d = (x % (D / 4)) * 4;
      if (i >= runs * QUADS) break;
      const unsigned mm = head->run[rn].members;
      const int e0 = __ffs(mm) - 1, e1 = __ffs(mm & (mm - 1)) - 1;
      w[u][0] = head->weight[hl * 32 + e0];
      w[u][1] = e1 < 0 ? 0.f : head->weight[hl * 32 + e1];
      p[u][0] = *reinterpret_cast<const float4 *>(record(e0) + hl * D + d);
      p[u][1] = e1 < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4 *>(record(e1) + hl * D + d);
    }
#pragma unroll
    for (int u = 0; u < FOUR; ++u) {
      const int i = i0 + u * THREADS, rn = i / QUADS, x = i - rn * QUADS, hl = x / (D / 4), d = (x % (D / 4)) * 4;
      if (i >= runs * QUADS) break;
      const AttnRun run = head->run[rn];
      float4 v;
      v.x = w[u][0] * p[u][0].x + w[u][1] * p[u][1].x;
      v.y = w[u][0] * p[u][0].y + w[u][1] * p[u][1].y;
      v.z = w[u][0] * p[u][0].z + w[u][1] * p[u][1].z;
      v.w = w[u][0] * p[u][0].w + w[u][1] * p[u][1].w;
      unsigned mm = run.members & (run.members - 1);
#pragma unroll 2
      for (mm &= mm - 1; mm; mm &= mm - 1) {
        const int e = __ffs(mm) - 1;
        const float we = head->weight[hl * 32 + e];
        const float4 pe = *reinterpret_cast<const float4 *>(record(e) + hl * D + d);
        v.x += we * pe.x; v.y += we * pe.y; v.z += we * pe.z; v.w += we * pe.w;
      }
      // (a run is its start's lane: the item's first segment, or lane 0 where it began before)
      const float lse2 = head->run_lse[hl * 32 + (run.begins ? run.first : 0)];
      if (run.begins && run.ends) {
        finish(head->seg[run.first], hl, d, v, lse2);
      } else {
        float *to = a.parts + ((size_t)blockIdx.x * 2 + run.begins) * (PART / 4);
        __stcg(reinterpret_cast<float4 *>(to + hl * D + d), v);
        if (d == 0) __stcg(to + GT * D + hl * 4, lse2);
      }
    }
  }

  // Items that span CTAs: the last CTA to arrive joins their records.  The
  // counter is that of the CTA in which the item begins.
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const AttnRun run = head->run[k ? max(runs - 1, 0) : 0];
      const bool spans = runs > 0 && !(run.begins && run.ends) && run.begins == k;
      int last = 0;
      if (spans) {
        const AttnSeg sg = head->seg[run.first];
        const int c0 = line.part_of(sg.start), n = line.part_of(sg.start + sg.nu - 1) - c0 + 1;
        s_from[k] = c0;
        s_from[2 + k] = n;
        s_from[4 + k] = run.first;
        // releases the CTA's records (ordered before by the barrier) and, for the last, acquires the others'
        if (atom_add_acq_rel(&a.counters[c0], 1) == n - 1) {
          a.counters[c0] = 0;
          last = 1;
        }
      }
      s_last[k] = last;
    }
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) {
    if (!s_last[k]) continue;
    const AttnSeg sg = head->seg[s_from[4 + k]];
    const int n = s_from[2 + k];
    // the records: that of the CTA in which the item begins, then the others'
    const float *recs = a.parts + (size_t)s_from[k] * 2 * (PART / 4);
    // Records come from the L2 that another SM wrote, thousands of cycles away:
    // sixteen pieces at a time are on their way, of as many quads as a thread has.
    constexpr int MINE = QUADS > THREADS ? (QUADS + THREADS - 1) / THREADS : 1, AHEAD = 16 / MINE;
    float m[MINE], s[MINE];
    float4 v[MINE];
#pragma unroll
    for (int u = 0; u < MINE; ++u) {
      m[u] = -INFINITY;
      s[u] = 0.f;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto quad = [&](int u) { return min(tid + u * THREADS, QUADS - 1); };
    for (int c0 = 0; c0 < n; c0 += AHEAD) {  // under a running reference
      float ls[MINE][AHEAD];
      float4 p[MINE][AHEAD];
#pragma unroll
      for (int u = 0; u < MINE; ++u)
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const int x = quad(u), c = c0 + j;
          const float *rec = recs + ((size_t)c * 2 + (c == 0 ? 1 : 0)) * (PART / 4);
          ls[u][j] = -INFINITY;
          p[u][j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < n) {
            ls[u][j] = __ldcg(rec + GT * D + x / (D / 4) * 4);
            p[u][j] = __ldcg(reinterpret_cast<const float4 *>(rec + x * 4));
          }
        }
#pragma unroll
      for (int u = 0; u < MINE; ++u) {
        float top = m[u];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) top = fmaxf(top, ls[u][j]);
        const float r = top == -INFINITY ? 0.f : top, keep = ex2(m[u] - r);
        m[u] = top;
        s[u] *= keep;
        v[u].x *= keep; v[u].y *= keep; v[u].z *= keep; v[u].w *= keep;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const float w = ex2(ls[u][j] - r);
          s[u] += w;
          v[u].x += w * p[u][j].x; v[u].y += w * p[u][j].y; v[u].z += w * p[u][j].z; v[u].w += w * p[u][j].w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < MINE; ++u) {
      const int x = tid + u * THREADS;
      if (x >= QUADS) break;
      const float inv = s[u] == 0.f ? 0.f : 1.f / s[u], lse2 = s[u] == 0.f ? -INFINITY : m[u] + lg2(s[u]);
      finish(sg, x / (D / 4), (x % (D / 4)) * 4, make_float4(v[u].x * inv, v[u].y * inv, v[u].z * inv, v[u].w * inv), lse2);
    }
  }
}

// Eight-head tiles per item: a second one from nine query heads per kv head
// on, so that the cache is read once for up to 16; larger groups read it once
// per 16 heads, mostly from L2.
static int attn_tiles(int group) { return group <= 8 ? 1 : 2; }

size_t attn_workspace_bytes(int fmt, int D, int group, int sms) {
  size_t n = 0;
  kv_dispatch(fmt, D, [&](auto F, auto DD) {
    n = attn_tiles(group) == 1 ? AttnShape<F, DD, 1>::workspace(sms) : AttnShape<F, DD, 2>::workspace(sms);
    return HQ_OK;
  });
  return align_up((size_t)sms * sizeof(int), 256) + n;
}

template <int FMT, int D, int NT>
static hq_status attn_start(const AttnArgs &a, int sms, cudaStream_t st) {
  using S = AttnShape<FMT, D, NT>;
  static std::atomic<unsigned> configured{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return HQ_ERR_CUDA;
  if (dev >= 32 || !(configured.load(std::memory_order_acquire) & (1u << dev))) {
    if (cudaFuncSetAttribute(attn_kernel<FMT, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) != cudaSuccess)
      return HQ_ERR_CUDA;
    if (dev < 32) configured.fetch_or(1u << dev, std::memory_order_release);
  }
  attn_kernel<FMT, D, NT><<<sms, (S::W + S::P) * 32, S::SMEM, st>>>(a);
  return check_launch();
}

hq_status launch_attn(int fmt, int D, AttnArgs a, int sms, void *workspace, cudaStream_t st) {
  const int nt = attn_tiles(a.group);
  a.hgroups = (a.group + 8 * nt - 1) / (8 * nt);
  a.counters = (int *)workspace;
  a.parts = (float *)((uint8_t *)workspace + align_up((size_t)sms * sizeof(int), 256));
  return kv_dispatch(fmt, D, [&](auto F, auto DD) {
    return nt == 1 ? attn_start<F, DD, 1>(a, sms, st) : attn_start<F, DD, 2>(a, sms, st);
  });
}

}  // namespace hq
