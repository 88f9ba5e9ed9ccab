// Rotary positions and the paged key-value cache: the rotation table, the
// rotation, the quantising write and the read back.
//
// Cache layout.  A page holds `page_size` tokens of every kv head:
//   [heads][page_size / 16] units, one unit = 16 consecutive tokens of one head:
//     [K codes][V codes][K scales][V scales]
// so a unit is one contiguous piece of HBM that a single bulk copy brings in.
// The codes are stored as the attention kernel's 32 lanes consume them (the A
// fragments of a 16 x 16 x 16 MMA whose M side is the tokens for K and the
// channels for V).  The grain is an octet, 8 consecutive channels of one
// token (GS = 16, 8 or 4 bytes); every lane owns D / 16 octets of K and D / 16
// of V, its octets are laid out in 16-byte vectors, and vector v of all
// 32 lanes is one conflict-free 512-byte shared-memory load:
//   byte(lane, i) = ((i * GS / 16) * 32 + lane) * 16 + (i * GS) % 16
//   K octet o of token r:  lane (r % 8) * 4 + o % 4,  i = (o / 4) * 2 + r / 8
//   V octet o of token r:  lane (o / (D / 64)) * 4 + (r % 8) / 2,
//                          i = (o % (D / 64)) * 4 + (r / 8) * 2 + r % 2
// Scales: E4M3 fp32 [16 tokens] for K, then V; NVFP4 K [16 tokens][2][D / 32]
// (16-channel block 2b + h at [h][b]), V [D / 16 blocks][16 tokens].
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "hq_internal.cuh"

namespace hq {

// ---- the rotation table ------------------------------------------------------
// Frequency i of a rotation of R channels, radians per position, in 64 bits.
__device__ __forceinline__ double rope_freq(const hq_rope_desc &d, int i) {
  const double two_pi = 6.283185307179586476925;
  double f = pow(d.base, -2.0 * i / d.rot_dim);
  if (d.scaling == HQ_ROPE_LINEAR) f /= d.factor;
  if (d.scaling == HQ_ROPE_TURNS) {
    const double turns = d.context * f / two_pi;
    const double y = fmin(fmax((turns - d.low) / (d.high - d.low), 0.0), 1.0);
    f = f * (y + (1.0 - y) / d.factor);
  }
  if (d.scaling == HQ_ROPE_INDEX) {
    // index of the frequency that makes n turns over the context
    const double den = 2.0 * log(d.base);
    const double at_high = d.rot_dim * log(d.context / (two_pi * d.high)) / den;
    const double at_low = d.rot_dim * log(d.context / (two_pi * d.low)) / den;
    const double first = fmax(floor(at_high), 0.0), last = fmin(ceil(at_low), d.rot_dim - 1.0);
    const double y = 1.0 - fmin(fmax((i - first) / fmax(last - first, 0.001), 0.0), 1.0);
    f = f * (y + (1.0 - y) / d.factor);
  }
  return f;
}

// amplitude * (cosine, sine) of a 64-bit fraction of a turn, within an fp32
// step of the value.  Whole quarters come off (Q); what is left, in units of
// 2^-32 of a turn, is t + d: t a multiple of 32 that fp32 holds, d the rest with
// 27 bits behind the point, so that small angles keep their bits.  r is the
// rounded t in radians and e what r lacks of the angle.  The polynomials are
// minimax fits for |r| <= pi / 4 (a linear program over 4001 points), off by
// 5.5e-9 of the sine and 6e-10, a tenth of a step; sine and cosine go on as r + u
// and 1 + w, and the product with the amplitude (amp + amp_rest) is rounded
// where the large part comes in.
__device__ __forceinline__ void turn_cos_sin(unsigned long long turn, float amp, float amp_rest, float &co, float &si) {
  const uint32_t hi = (uint32_t)(turn >> 32), lo = (uint32_t)turn, Q = (hi + (1u << 29)) & 0xC0000000u;
  const uint32_t h = hi - Q + 16u;
  const float t = (float)(int)(h & ~31u), d = (float)(int)(((h << 27) | (lo >> 5)) ^ 0x80000000u);
  constexpr float C = 6.283185307179586f / 4294967296.f;  // radians a unit, and what it lacks
  constexpr float C_REST = (float)(6.283185307179586 / 4294967296.0 - (double)C);
  const float r = t * C, e = fmaf(d, C / 134217728.f, fmaf(t, C_REST, fmaf(t, C, -r)));
  const float z = r * r;
  const float p = fmaf(fmaf(z, -1.9517266e-4f, 8.332178e-3f), z, -1.6666655e-1f);                 // (sin r - r) / r^3
  const float q = fmaf(fmaf(fmaf(z, 2.4438406e-5f, -1.3887368e-3f), z, 4.1666646e-2f), z, -0.5f);  // (cos r - 1) / r^2
  const float u = fmaf(p * z, r, e), w = fmaf(q, z, -e * r);
  const float s = fmaf(amp, r, fmaf(amp, u, amp_rest * r)), c = amp + fmaf(amp, w, amp_rest);
  const bool odd = Q & 0x40000000u;
  si = __uint_as_float(__float_as_uint(odd ? c : s) ^ (Q & 0x80000000u));
  co = __uint_as_float(__float_as_uint(odd ? s : c) ^ ((Q + 0x40000000u) & 0x80000000u));
}

// table[p] = amplitude * (cos(p f_0) .. cos(p f_{R/2-1}), sin(p f_0) ..).  The
// angle of a far position does not fit fp32 (position 131072 leaves 2^-7 of a
// radian there).  It is counted in turns, as a 64-bit binary fraction per
// position (2^-53 of the frequency, 2^-64 of a turn), whose product with p
// drops whole turns by itself.  131072 x 128 (67 MB) takes 14.6 us of a floor of
// 10.2: 3 until the blocks have their frequencies (64-bit powers), then some 45
// instructions an angle beside the stores (64-bit floating point in the loop:
// 21).  The powers take 64 registers, so four blocks an SM are resident; a
// grid of twice that computes the frequencies a second time behind them: 16.5.
constexpr int TABLE_THREADS = 256, TABLE_BLOCKS = 4;  // of an SM
template <int V>
__global__ void __launch_bounds__(TABLE_THREADS, TABLE_BLOCKS) rope_table_kernel(hq_rope_desc d, int P, float *__restrict__ table) {
  __shared__ unsigned long long per[512];  // turns per position, times 2^64
  const int half = d.rot_dim / 2;
  const float amp = (float)d.amplitude, amp_rest = (float)(d.amplitude - (double)amp);
  for (int i = threadIdx.x; i < half; i += TABLE_THREADS) {
    const double turns = rope_freq(d, i) / 6.283185307179586476925;
    per[i] = (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0);
  }
  __syncthreads();
  // Threads of a block: `cols` sets of V neighbouring frequencies (all, up to
  // the block's width) x rows.
  const int sets = half / V, cols = min(sets, TABLE_THREADS), rows = TABLE_THREADS / cols;
  const int row = threadIdx.x / cols;
  if (row >= rows) return;
  for (int i = (threadIdx.x - row * cols); i < sets; i += cols) {
    unsigned long long f[V];
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = per[i * V + j];
    const unsigned step = gridDim.x * rows;
    float *to = table + (size_t)(blockIdx.x * rows + row) * d.rot_dim + i * V;
    for (unsigned p = blockIdx.x * rows + row; p < (unsigned)P; p += step, to += (size_t)step * d.rot_dim) {
      float co[V], si[V];
#pragma unroll
      for (int j = 0; j < V; ++j) turn_cos_sin(f[j] * p, amp, amp_rest, co[j], si[j]);
      if constexpr (V == 4) {
        __stcs(reinterpret_cast<float4 *>(to), make_float4(co[0], co[1], co[2], co[3]));
        __stcs(reinterpret_cast<float4 *>(to + half), make_float4(si[0], si[1], si[2], si[3]));
      } else {
        to[0] = co[0];
        to[half] = si[0];
      }
    }
  }
}

hq_status launch_rope_table(const hq_rope_desc *d, int P, float *table, cudaStream_t st) {
  hq_rope_desc r = *d;
  if (r.amplitude == 0.0) r.amplitude = 1.0;
  const int half = r.rot_dim / 2, v = half % 4 == 0 ? 4 : 1, sets = half / v;
  const int rows = TABLE_THREADS / (sets < TABLE_THREADS ? sets : TABLE_THREADS);
  const int want = P / rows + (P % rows != 0), most = 148 * TABLE_BLOCKS, blocks = want < most ? want : most;
  if (v == 4) rope_table_kernel<4><<<blocks, TABLE_THREADS, 0, st>>>(r, P, table);
  else rope_table_kernel<1><<<blocks, TABLE_THREADS, 0, st>>>(r, P, table);
  return check_launch();
}

// ---- the rotation --------------------------------------------------------------
// (a, b) -> (a c - b s, b c + a s), each step an fp32 IEEE operation.
__device__ __forceinline__ void rope_pair(float a, float b, float c, float s, float &x, float &y) {
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

__device__ __forceinline__ float bf16_at(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ uint16_t to_bf16(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  return (uint32_t)to_bf16(lo) | ((uint32_t)to_bf16(hi) << 16);
}
__device__ __forceinline__ void unpack8(const uint4 v, float *f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float *f) {
  return make_uint4(to_bf16x2(f[0], f[1]), to_bf16x2(f[2], f[3]), to_bf16x2(f[4], f[5]), to_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float *p, float *f) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Work of a head.  Interleaved pairs, and halves of a multiple of 8: chunks of
// 8 pairs, then chunks of 16 unrotated channels (the last may have 8; the last
// of interleaved pairs may end with unrotated channels).  Halves of another
// width, whose pairs straddle 16-byte pieces: single pairs, then two unrotated
// channels at a time, neighbours to neighbouring lanes.  Both channels of a
// pair are one thread's, so x and out may be the same.
enum RopeWidth { ROPE_EVEN, ROPE_RAGGED, ROPE_SINGLE };
__host__ __device__ inline RopeWidth rope_width(int rot, int inter) {
  return rot % 16 == 0 ? ROPE_EVEN : inter ? ROPE_RAGGED : ROPE_SINGLE;
}
inline int rope_pairs(int rot, int inter) { return rope_width(rot, inter) == ROPE_SINGLE ? rot / 2 : (rot + 15) / 16; }
inline int rope_rest(int D, int rot, int inter) {
  if (rope_width(rot, inter) == ROPE_SINGLE) return (D - rot) / 2;
  const int left = D - 16 * rope_pairs(rot, inter);
  return left > 0 ? (left + 15) / 16 : 0;
}

// A chunk is two 16-byte pieces (the second may be missing), loaded before
// anything that depends on the position.
struct RopePiece {
  const uint16_t *x;  // the head's row
  uint16_t *out;
  int c, p;           // chunk (or pair), position
  uint4 a, b;
};
template <RopeWidth W>
__device__ __forceinline__ void rope_where(const RopePiece &r, int D, int rot, int inter, int &i0, int &i1, bool &pair) {
  if constexpr (W == ROPE_RAGGED) {
    pair = r.c < (rot + 15) / 16;
    i0 = 16 * r.c;
    i1 = i0 + 8 < D ? i0 + 8 : -1;
    return;
  }
  const int half = rot / 2, npair = half / 8;
  pair = r.c < npair;
  if (pair) {
    i0 = inter ? 16 * r.c : 8 * r.c;
    i1 = inter ? i0 + 8 : i0 + half;
  } else {
    i0 = rot + 16 * (r.c - npair);
    i1 = i0 + 8 < D ? i0 + 8 : -1;
  }
}
template <RopeWidth W>
__device__ __forceinline__ void rope_piece(const RopePiece &r, int D, int rot, int inter, const float *tab) {
  int i0, i1;
  bool pair;
  rope_where<W>(r, D, rot, inter, i0, i1, pair);
  if (!pair) {
    if (r.x == r.out) return;
    __stcs(reinterpret_cast<uint4 *>(r.out + i0), r.a);
    if (i1 >= 0) __stcs(reinterpret_cast<uint4 *>(r.out + i1), r.b);
    return;
  }
  float a[8], b[8], co[8], si[8];
  unpack8(r.a, a);
  unpack8(r.b, b);
  const int half = rot / 2;
  if constexpr (W == ROPE_RAGGED) {  // rows of the table are not 16-byte aligned
    const int n = half - 8 * r.c;    // pairs that are rotated
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      co[j] = j < n ? tab[8 * r.c + j] : 0.f;
      si[j] = j < n ? tab[half + 8 * r.c + j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < n) rope_pair(a[2 * j], a[2 * j + 1], co[j], si[j], a[2 * j], a[2 * j + 1]);
      if (4 + j < n) rope_pair(b[2 * j], b[2 * j + 1], co[4 + j], si[4 + j], b[2 * j], b[2 * j + 1]);
    }
  } else {
    load8(tab + 8 * r.c, co);
    load8(tab + half + 8 * r.c, si);
    if (inter) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        rope_pair(a[2 * j], a[2 * j + 1], co[j], si[j], a[2 * j], a[2 * j + 1]);
        rope_pair(b[2 * j], b[2 * j + 1], co[4 + j], si[4 + j], b[2 * j], b[2 * j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) rope_pair(a[j], b[j], co[j], si[j], a[j], b[j]);
    }
  }
  __stcs(reinterpret_cast<uint4 *>(r.out + i0), pack8(a));
  if (W == ROPE_EVEN || i1 >= 0) __stcs(reinterpret_cast<uint4 *>(r.out + i1), pack8(b));
}

// n / d for n < 2^31 by a product: q = (umulhi(n, m) + n) >> s with
// s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1.
struct FastDiv {
  uint32_t d, m;
  int s;
};
static FastDiv fast_div(uint32_t d) {
  int s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{d, (uint32_t)(((((1ull << s) - d) << 32) / d) + 1), s};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) { return (__umulhi(n, f.m) + n) >> f.s; }

struct RopeArgs {
  int T, H, D, rot, inter, P;
  const uint16_t *x;
  long long xt, xh;  // strides between tokens and heads, elements
  const int32_t *pos;
  const float *table;
  uint16_t *out;
  long long ot, oh;
  FastDiv pairs, rest, per_token;  // chunks with and without pairs of a head, chunks of a token
  FastDiv parts;              // blocks of a token
  int tokens;                 // tokens of a block
};

// A block has a chunk, or ROPE_NARROW single pairs, a thread: of several whole
// tokens, or one of `parts` parts of a token.
constexpr int ROPE_NARROW = 8;
struct RopeSplit {
  int tokens, parts;
};
inline RopeSplit rope_split(int T, int per_token, int full) {
  int n = full / per_token;
  if (n > T / (148 * 4)) n = T / (148 * 4);  // blocks enough for every SM come first
  return RopeSplit{n > 1 ? n : 1, (per_token + full - 1) / full};
}
inline long long rope_blocks(const RopeArgs &a) { return ((long long)a.T + a.tokens - 1) / a.tokens * a.parts.d; }

// Bound by HBM: x is read and out written once, the table rows come from L2
// (one of a token for all of its heads).  8191 tokens x 32 heads x 192 (a third
// rotated): 37.0 us, 5.5 TB/s of the measured 6.55.  One chunk a thread and 24
// warps an SM beat two to four chunks (42 to 49 us), streaming loads and stores
// (they are used once) plain ones (39.6), blocks of 128 those of 256 (37.6).
// Of 136 rotated (3625 x 64 x 192, a floor of 27 us) interleaved pairs take 36,
// in single pairs 89; halves take 75, in single pairs bound by their
// instructions, and in chunks of eight read channel by channel 228.  A kernel
// for each width: sharing one, the ragged code cost the even widths 6%.
template <RopeWidth W>
__device__ __forceinline__ void rope_rows(const RopeArgs &a, uint32_t block) {
  const uint32_t tb = div_by(block, a.parts), part = block - tb * a.parts.d;
  const long long t0 = (long long)tb * a.tokens;
  const uint32_t n = (uint32_t)min((long long)a.tokens, a.T - t0) * a.per_token.d, np = a.H * a.pairs.d;
  // item i of the block: a token's pairs come first, head by head, then the
  // rest, so that warps rarely do both
  auto locate = [&](uint32_t i, RopePiece &r) {
    const uint32_t tt = div_by(i, a.per_token), in = i - tt * a.per_token.d;
    const uint32_t j = in < np ? in : in - np, h = div_by(j, in < np ? a.pairs : a.rest);
    const long long t = t0 + tt;
    r.c = in < np ? j - h * a.pairs.d : a.pairs.d + j - h * a.rest.d;
    r.p = a.pos[t];
    r.x = a.x + t * a.xt + h * a.xh;
    r.out = a.out + t * a.ot + h * a.oh;
  };
  auto known = [&](int p) {
    if (p >= 0 && p < a.P) return true;
    set_device_error(HQ_ERR_DEVICE_INDEX);
    return false;
  };
  if constexpr (W != ROPE_SINGLE) {
    const uint32_t i = part * blockDim.x + threadIdx.x;
    if (i >= n) return;
    RopePiece r;
    locate(i, r);
    int p0, p1;
    bool pair;
    rope_where<W>(r, a.D, a.rot, a.inter, p0, p1, pair);
    if (!pair && r.x == r.out) return;
    r.a = __ldcs(reinterpret_cast<const uint4 *>(r.x + p0));
    if (p1 >= 0) r.b = __ldcs(reinterpret_cast<const uint4 *>(r.x + p1));
    if (known(r.p)) rope_piece<W>(r, a.D, a.rot, a.inter, a.table + (size_t)r.p * a.rot);
    return;
  }
  const int half = a.rot / 2;
#pragma unroll 4
  for (int u = 0; u < ROPE_NARROW; ++u) {
    const uint32_t i = (part * ROPE_NARROW + u) * blockDim.x + threadIdx.x;
    if (i >= n) break;
    RopePiece r;
    locate(i, r);
    if (!known(r.p)) continue;
    if (r.c >= half) {
      const int ch = a.rot + 2 * (r.c - half);
      *reinterpret_cast<uint32_t *>(r.out + ch) = *reinterpret_cast<const uint32_t *>(r.x + ch);
      continue;
    }
    const float *tab = a.table + (size_t)r.p * a.rot;
    const float co = tab[r.c], si = tab[half + r.c];
    float v, w;
    rope_pair(bf16_at(r.x + r.c), bf16_at(r.x + r.c + half), co, si, v, w);
    r.out[r.c] = to_bf16(v);
    r.out[r.c + half] = to_bf16(w);
  }
}

constexpr int ROPE_THREADS = 128;
template <RopeWidth W>
__global__ void __launch_bounds__(ROPE_THREADS, W == ROPE_EVEN ? 12 : W == ROPE_RAGGED ? 10 : 8) rope_kernel(RopeArgs a) {
  rope_rows<W>(a, blockIdx.x);
}

RopeArgs rope_args(int T, int H, int D, const hq_rope_desc *r, int P, const void *x, int64_t xt, int64_t xh,
                   const int32_t *pos, const float *table, void *out, int64_t ot, int64_t oh, int threads) {
  const int pairs = rope_pairs(r->rot_dim, r->interleaved), rest = rope_rest(D, r->rot_dim, r->interleaved);
  const int per_token = (pairs + rest) * (H > 0 ? H : 1);
  const RopeSplit split = rope_split(T, per_token, rope_width(r->rot_dim, r->interleaved) == ROPE_SINGLE ? threads * ROPE_NARROW : threads);
  return RopeArgs{T, H, D, r->rot_dim, r->interleaved, P, (const uint16_t *)x, xt, xh, pos, table, (uint16_t *)out,
                  ot, oh, fast_div(pairs), fast_div(rest > 0 ? rest : 1), fast_div(per_token), fast_div(split.parts), split.tokens};
}

hq_status launch_rope(const RopeArgs &a, cudaStream_t st) {
  const RopeWidth w = rope_width(a.rot, a.inter);
  auto *const kernel = w == ROPE_EVEN ? rope_kernel<ROPE_EVEN> : w == ROPE_RAGGED ? rope_kernel<ROPE_RAGGED> : rope_kernel<ROPE_SINGLE>;
  kernel<<<(unsigned)rope_blocks(a), ROPE_THREADS, 0, st>>>(a);
  return check_launch();
}

// ---- the cache layout ------------------------------------------------------------
__host__ __device__ constexpr int kv_granule(int fmt) { return fmt == A_BF16 ? 16 : fmt == A_FP8 ? 8 : 4; }
__host__ __device__ constexpr int kv_code_bytes(int fmt, int D) { return 2 * D * kv_granule(fmt); }  // 16 tokens of K or V
__host__ __device__ constexpr int kv_scale_bytes(int fmt, int D) { return fmt == A_BF16 ? 0 : fmt == A_FP8 ? 64 : D; }
__host__ __device__ constexpr int kv_unit_bytes(int fmt, int D) {
  return 2 * (kv_code_bytes(fmt, D) + kv_scale_bytes(fmt, D));
}

template <int GS>
__device__ __forceinline__ int lane_byte(int lane, int i) {
  return ((i * GS / 16) * 32 + lane) * 16 + (i * GS) % 16;
}
template <int GS>
__device__ __forceinline__ int k_octet(int o, int r) {
  return lane_byte<GS>((r & 7) * 4 + (o & 3), (o >> 2) * 2 + (r >> 3));
}
template <int GS, int D>
__device__ __forceinline__ int v_octet(int o, int r) {
  constexpr int NQ = D / 64;
  return lane_byte<GS>((o / NQ) * 4 + ((r & 7) >> 1), (o % NQ) * 4 + (r >> 3) * 2 + (r & 1));
}

struct KvArgs {
  int H, page_units;        // kv heads; units per page
  int page;                 // tokens per page
  long long slots_total;    // num_pages * page
  size_t page_bytes;
  uint8_t *pages;
  const float *glob;        // NVFP4: second-level scales of K and V
};

// Octet o of a row, rotated in fp32; any width, channel by channel.
__device__ __noinline__ void rope_octet_slow(const uint16_t *x, int o, int rot, int inter, const float *tab, float *f) {
  const int half = rot / 2;
  for (int i = 0; i < 8; ++i) {
    const int ch = 8 * o + i;
    f[i] = bf16_at(x + ch);
    if (ch >= rot) continue;
    const int j = inter ? ch >> 1 : (ch < half ? ch : ch - half);
    const bool second = inter ? (ch & 1) : ch >= half;
    const float other = bf16_at(x + (inter ? ch ^ 1 : second ? ch - half : ch + half));
    float u;
    if (second) rope_pair(other, f[i], tab[j], tab[half + j], u, f[i]);
    else rope_pair(f[i], other, tab[j], tab[half + j], f[i], u);
  }
}

__device__ __forceinline__ void rope_octet(const uint16_t *x, int o, int rot, int inter, const float *tab, float *f) {
  const int half = rot / 2, ch = 8 * o;
  if (rot & 15) {
    float tmp[8];
    rope_octet_slow(x, o, rot, inter, tab, tmp);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = tmp[i];
    return;
  }
  unpack8(*reinterpret_cast<const uint4 *>(x + ch), f);
  if (ch >= rot) return;
  if (inter) {  // the pairs are within the octet
    const float4 co = *reinterpret_cast<const float4 *>(tab + ch / 2), si = *reinterpret_cast<const float4 *>(tab + half + ch / 2);
    rope_pair(f[0], f[1], co.x, si.x, f[0], f[1]);
    rope_pair(f[2], f[3], co.y, si.y, f[2], f[3]);
    rope_pair(f[4], f[5], co.z, si.z, f[4], f[5]);
    rope_pair(f[6], f[7], co.w, si.w, f[6], f[7]);
  } else {
    const bool second = ch >= half;
    const int j = second ? ch - half : ch;
    float p[8], co[8], si[8];
    unpack8(*reinterpret_cast<const uint4 *>(x + (second ? j : ch + half)), p);
    load8(tab + j, co);
    load8(tab + half + j, si);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // a c - b s for the first of a pair, b c + a s for the second
      const float u = __fmul_rn(f[i], co[i]), v = __fmul_rn(p[i], si[i]);
      f[i] = second ? __fadd_rn(u, v) : __fsub_rn(u, v);
    }
  }
}

struct KvRows {
  int T;
  const uint16_t *k, *v;
  long long ks, vs;         // strides between tokens, elements
  const long long *slots;
  uint16_t *k_out, *v_out;  // read back
};

// A warp writes (reads) 16 consecutive tokens of the call and one head, its
// lanes in the layout's own order: lane (g, t) = 4 g + t has octets 4 b + t of
// keys g and g + 8 and octets g (D / 64) + q of values 2t, 2t + 1, 2t + 8,
// 2t + 9, which are exactly the 16-byte vectors it holds in a unit.  Where the
// tokens' slots run through one unit, or through the end of one and the
// beginning of another (a prompt: rows r0, r0 + 1, .. modulo 16), lanes go by
// the row in the unit and move whole vectors (split where their octets are in
// two units); other groups (a decoding step's tokens) go by the token and move
// octet by octet.  No shared memory, no barrier.
constexpr int KV_THREADS = 128;

struct KvGroup {
  long long unit;  // lane i (and i + 16): byte offset of token i's unit (head 0), -1: none
  int row, pos;    // and its position
  bool run;
  int r0;
};
struct KvToken {   // what a lane reads of its token
  long long slot;
  int pos;
};
__device__ __forceinline__ KvToken kv_token(const KvRows &w, const RopeArgs *rope, long long t0) {
  const long long t = t0 + (threadIdx.x & 15);
  return t < w.T ? KvToken{w.slots[t], rope ? rope->pos[t] : 0} : KvToken{-1, 0};
}

template <int FMT, int D>
__device__ __forceinline__ KvGroup kv_group(const KvArgs &a, const KvToken &k, const RopeArgs *rope) {
  const int i = threadIdx.x & 15;
  KvGroup s{-1, 0, k.pos, false, 0};
  if (k.slot >= a.slots_total) set_device_error(HQ_ERR_DEVICE_INDEX);
  if (k.slot >= 0 && k.slot < a.slots_total) {
    const long long pg = k.slot >> 31 ? k.slot / a.page : (long long)((uint32_t)k.slot / (uint32_t)a.page);
    const int off = (int)(k.slot - pg * a.page);
    s.unit = (long long)((size_t)pg * a.page_bytes + (size_t)(off >> 4) * kv_unit_bytes(FMT, D));
    s.row = off & 15;
    if (rope && (k.pos < 0 || k.pos >= rope->P)) {
      set_device_error(HQ_ERR_DEVICE_INDEX);
      s.unit = -1;
    }
  }
  const int r0 = __shfl_sync(0xffffffffu, s.row, 0);
  const long long u0 = __shfl_sync(0xffffffffu, s.unit, 0), u1 = __shfl_sync(0xffffffffu, s.unit, 15);
  s.run = __all_sync(0xffffffffu, s.unit >= 0 && s.row == ((r0 + i) & 15) && s.unit == (r0 + i < 16 ? u0 : u1));
  s.r0 = s.run ? r0 : 0;
  return s;
}

// One of a lane's rows: the token of the call, and where it is held.
struct KvRow {
  int i, row;
  long long unit;
};
__device__ __forceinline__ KvRow kv_row(const KvGroup &s, int r) {  // r: the lane's row in the layout
  KvRow k;
  k.i = (r - s.r0) & 15;
  k.unit = __shfl_sync(0xffffffffu, s.unit, k.i);
  k.row = __shfl_sync(0xffffffffu, s.row, k.i);
  return k;
}

__device__ __forceinline__ float amax8(const float *f) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}
// hq_quant_act's per-token recipe on a head's D channels
// (rotated channels reach below bf16's smallest number, where the quotient may be 0)
__device__ __forceinline__ float e4m3_scale(float amax) {
  const float s = __fdiv_rn(amax, 448.f);
  return s == 0.f ? 1.f : s;
}
// Correctly rounded quotients by one divisor, by Markstein's theorem ("Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990): with
// y the correctly rounded 1 / d and q within one step of x / d, r = x - q d is
// exact in an fma and q + r y, rounded, is the correctly rounded x / d, as
// long as nothing over- or underflows.  y and the rest of 1 / d make a first
// q that is off by little more than half a step.  Four instructions and the
// sign (a zero keeps it) instead of a division each.  Rows whose divisor or
// largest element is out of range divide.  (Dividends too small for an exact
// r have quotients far under half of the smallest code.)
struct Divisor {
  float d, y, rest;
  bool plain;
};
__device__ __forceinline__ Divisor divisor(float d, float amax) {
  const float y = __frcp_rn(d);
  return Divisor{d, y, __fmul_rn(__fmaf_rn(-d, y, 1.f), y), !(d > 1e-18f && d < 1e18f && amax < 1e18f)};
}
__device__ __forceinline__ float quotient(float x, const Divisor &v) {  // not v.plain
  const float q = __fmaf_rn(x, v.y, __fmul_rn(x, v.rest));
  return copysignf(__fmaf_rn(__fmaf_rn(-q, v.d, x), v.y, q), x);
}
// Four codes a word.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{.reg .b16 l,h; cvt.rn.satfinite.e4m3x2.f32 l, %2, %1; cvt.rn.satfinite.e4m3x2.f32 h, %4, %3; mov.b32 %0, {l,h};}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint32_t e2m1x8(const float *f) {
  uint32_t r;
  asm("{.reg .b8 a,b,c,d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a,b,c,d};}"
      : "=r"(r) : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
struct Octet {
  float f[8];
};
__device__ __noinline__ Octet octet_divided(Octet x, float d) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x.f[i] = __fdiv_rn(x.f[i], d);
  return x;
}
__device__ __forceinline__ Octet octet_quotients(const float *f, const Divisor &v) {
  Octet x;
  if (v.plain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.f[i] = f[i];
    return octet_divided(x, v.d);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x.f[i] = quotient(f[i], v);
  return x;
}
__device__ __forceinline__ uint2 e4m3_octet(const float *f, const Divisor &s) {
  const Octet x = octet_quotients(f, s);
  return make_uint2(e4m3x4(x.f[0], x.f[1], x.f[2], x.f[3]), e4m3x4(x.f[4], x.f[5], x.f[6], x.f[7]));
}
// hq_quant_act's NVFP4 recipe with a static tensor scale, on a block of 16
__device__ __noinline__ float nvfp4_scale_divided(float amax, float g) { return __fdiv_rn(__fdiv_rn(amax, 6.f), g); }
__device__ __forceinline__ uint32_t nvfp4_scale(float amax, const Divisor &g) {
  const Divisor six = divisor(6.f, 0.f);
  const float s = g.plain || !(amax < 1e18f) ? nvfp4_scale_divided(amax, g.d) : quotient(quotient(amax, six), g);
  return f32x2_to_e4m3x2(s, 0.f) & 0xFFu;
}
__device__ __forceinline__ uint32_t nvfp4_octet(const float *f, uint32_t sb, float g, float amax) {
  const float d = __fmul_rn(e4m3_to_f32(sb), g);
  if (d == 0.f) return 0;
  const Octet x = octet_quotients(f, divisor(d, amax));
  return e2m1x8(x.f);
}

// Warps that share the octets of a group and head: 64 channels each, but for
// E4M3, whose scale needs a whole row.
__host__ __device__ constexpr int kv_parts(int fmt, int D) { return fmt == A_FP8 ? 1 : D / 64; }

// Two warps a group, head and part, one for keys and one for values, each with
// a single item: what waits (slots, positions, then rows and table) is hidden
// by the number of warps, 32 an SM at 64 registers.  With rows in registers
// and everything unrolled, warps waited for instructions half of the time;
// with loops over octets or heads they were too few (8191 tokens x 4 heads x
// 256 with positions, NVFP4: 59, 28 and 30 us; this form: 21 of a floor of
// 7).  Its time goes to latency and to the recipe's arithmetic (some 200
// instructions per octet, the values' maxima and scales computed by both lanes
// of a block; the cap of 64 registers spills 36 to 80 bytes), bf16 rows' to
// latency alone.  8191 tokens, 32 + 8 heads x 128 with positions, and read
// back: bf16 66 us of a floor of 42, E4M3 87 of 37, NVFP4 65 of 34.
template <int FMT, int D, bool ROPE>
__global__ void __launch_bounds__(KV_THREADS, FMT != A_FP8 ? 8 : ROPE ? 4 : 6)
    kv_write_kernel(KvArgs a, KvRows w, RopeArgs rope, unsigned kv_blocks) {
  // The blocks past kv_blocks rotate the rope.H heads of q (mixed in between
  // the others, to copy beside the arithmetic, they took 12% more).
  if (blockIdx.x >= kv_blocks) {
    const RopeWidth w = rope_width(rope.rot, rope.inter);
    if (w == ROPE_EVEN) rope_rows<ROPE_EVEN>(rope, blockIdx.x - kv_blocks);
    else if (w == ROPE_RAGGED) rope_rows<ROPE_RAGGED>(rope, blockIdx.x - kv_blocks);
    else rope_rows<ROPE_SINGLE>(rope, blockIdx.x - kv_blocks);
    return;
  }
  constexpr int NB = D / 32, NQ = D / 64, CB = kv_code_bytes(FMT, D), SB = kv_scale_bytes(FMT, D), GS = kv_granule(FMT);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int PARTS = kv_parts(FMT, D);
  // the heads of a group are neighbours: they share the table's rows in L1
  const long long it = blockIdx.x * (long long)(KV_THREADS / 32) + (threadIdx.x >> 5), sets = it >> 31 ? it / a.H : (long long)((uint32_t)it / (uint32_t)a.H);
  const int h = (int)(it - sets * a.H), part = (int)((sets >> 1) % PARTS);
  const bool is_v = sets & 1;
  const long long t0 = (sets >> 1) / PARTS * 16;
  if (t0 < w.T) {
    const KvGroup s = kv_group<FMT, D>(a, kv_token(w, ROPE ? &rope : nullptr, t0), ROPE ? &rope : nullptr);
    uint8_t *base = a.pages + (size_t)h * a.page_units * kv_unit_bytes(FMT, D);

    if (!is_v) {
      KvRow kr[2];
      const uint16_t *x[2];
      const float *tab[2] = {nullptr, nullptr};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        kr[k] = kv_row(s, g + 8 * k);
        x[k] = w.k + (t0 + kr[k].i) * w.ks + (size_t)h * D;
        const int pos = __shfl_sync(0xffffffffu, s.pos, kr[k].i);
        if (ROPE && kr[k].unit >= 0) tab[k] = rope.table + (size_t)pos * rope.rot;
      }
      auto key = [&](int k, int b, float *f) {  // octet 4 b + t of key k as fp32
        if (kr[k].unit < 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = 0.f;
        } else if constexpr (ROPE) {
          rope_octet(x[k], 4 * b + t, rope.rot, rope.inter, tab[k], f);
        } else {
          unpack8(*reinterpret_cast<const uint4 *>(x[k] + 32 * b + 8 * t), f);
        }
      };
      const bool whole = s.run && kr[0].unit == kr[1].unit;
      if constexpr (FMT == A_BF16) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int b = 2 * part + j;
            uint4 v = make_uint4(0, 0, 0, 0);
            if constexpr (ROPE) {
              float f[8];
              key(k, b, f);
              v = pack8(f);
            } else if (kr[k].unit >= 0) {
              v = *reinterpret_cast<const uint4 *>(x[k] + 32 * b + 8 * t);
            }
            if (kr[k].unit >= 0) *reinterpret_cast<uint4 *>(base + kr[k].unit + k_octet<GS>(4 * b + t, kr[k].row)) = v;
          }
      } else if constexpr (FMT == A_FP8) {
        // Up to 128 channels a row is kept between the passes (without positions
        // 232 bytes of it in local memory: 80 registers for six blocks an SM).
        // Beyond, the second pass reads it again (from L1) and rotates it again,
        // in a loop that is not unrolled: the body would outgrow the instruction
        // cache.
        constexpr bool KEEP = D <= 128;
        float f[2][KEEP ? NB : 1][8], amax[2] = {0.f, 0.f};
        auto octet = [&](int k, int b) { return f[k][KEEP ? b : 0]; };
#pragma unroll(KEEP ? NB : 1)
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            key(k, b, octet(k, b));
            amax[k] = fmaxf(amax[k], amax8(octet(k, b)));
          }
        }
        Divisor sc[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          amax[k] = fmaxf(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], 1));
          amax[k] = fmaxf(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], 2));
          sc[k] = divisor(e4m3_scale(amax[k]), amax[k]);
          if (t == 0 && kr[k].unit >= 0) reinterpret_cast<float *>(base + kr[k].unit + 2 * CB)[kr[k].row] = sc[k].d;
        }
#pragma unroll(KEEP ? NB : 1)
        for (int b = 0; b < NB; ++b) {
          uint2 c[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (!KEEP) key(k, b, octet(k, b));
            c[k] = e4m3_octet(octet(k, b), sc[k]);
          }
          if (whole) {
            *reinterpret_cast<uint4 *>(base + kr[0].unit + (b * 32 + lane) * 16) = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (kr[k].unit >= 0) *reinterpret_cast<uint2 *>(base + kr[k].unit + k_octet<GS>(4 * b + t, kr[k].row)) = c[k];
          }
        }
      } else {
        const float gl = a.glob[0];
        const Divisor gd = divisor(gl, 0.f);
        const int b = 2 * part;
        uint32_t c[2][2], sb[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float f[8];
            key(k, b + j, f);
            float amax = amax8(f);
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            sb[j][k] = nvfp4_scale(amax, gd);
            c[j][k] = nvfp4_octet(f, sb[j][k], gl, amax);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k)  // the blocks of octets b and b + 1 are neighbours
          if ((t & 1) == 0 && kr[k].unit >= 0)
            *reinterpret_cast<uint16_t *>(base + kr[k].unit + 2 * CB + kr[k].row * (D / 16) + (t >> 1) * NB + b) =
                (uint16_t)(sb[0][k] | sb[1][k] << 8);
        if (whole) {
          *reinterpret_cast<uint4 *>(base + kr[0].unit + (b * 16 + lane) * 16) = make_uint4(c[0][0], c[0][1], c[1][0], c[1][1]);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (kr[k].unit >= 0)
                *reinterpret_cast<uint32_t *>(base + kr[k].unit + k_octet<GS>(4 * (b + j) + t, kr[k].row)) = c[j][k];
        }
      }
      return;
    }

    KvRow vr[4];
    const uint16_t *x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      vr[k] = kv_row(s, 2 * t + (k & 1) + 8 * (k >> 1));
      x[k] = w.v + (t0 + vr[k].i) * w.vs + (size_t)h * D;
    }
    auto value = [&](int k, int o) {  // octet o of value k
      return vr[k].unit >= 0 ? *reinterpret_cast<const uint4 *>(x[k] + 8 * o) : make_uint4(0, 0, 0, 0);
    };
    if constexpr (FMT == A_BF16) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 v = value(k, g * NQ + part);
        if (vr[k].unit >= 0)
          *reinterpret_cast<uint4 *>(base + vr[k].unit + CB + v_octet<GS, D>(g * NQ + part, vr[k].row)) = v;
      }
    } else if constexpr (FMT == A_FP8) {
      constexpr bool KEEP = D <= 128;  // as for the keys
      uint4 row[4][KEEP ? NQ : 1];
      float amax[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll(KEEP ? NQ : 1)
      for (int q = 0; q < NQ; ++q) {
#pragma unroll
        for (int k = 0; k < 4; ++k) row[k][KEEP ? q : 0] = value(k, g * NQ + q);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f[8];
          unpack8(row[k][KEEP ? q : 0], f);
          amax[k] = fmaxf(amax[k], amax8(f));
        }
      }
      Divisor sc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) amax[k] = fmaxf(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], o));
        sc[k] = divisor(e4m3_scale(amax[k]), amax[k]);
        if (g == 0 && vr[k].unit >= 0) reinterpret_cast<float *>(base + vr[k].unit + 2 * CB + SB)[vr[k].row] = sc[k].d;
      }
#pragma unroll(KEEP ? NQ : 1)
      for (int q = 0; q < NQ; ++q) {
        uint2 c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f[8];
          unpack8(KEEP ? row[k][KEEP ? q : 0] : value(k, g * NQ + q), f);
          c[k] = e4m3_octet(f, sc[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          if (s.run && vr[k].unit == vr[k + 1].unit) {
            *reinterpret_cast<uint4 *>(base + vr[k].unit + CB + ((q * 2 + k / 2) * 32 + lane) * 16) =
                make_uint4(c[k].x, c[k].y, c[k + 1].x, c[k + 1].y);
          } else {
#pragma unroll
            for (int j = k; j < k + 2; ++j)
              if (vr[j].unit >= 0)
                *reinterpret_cast<uint2 *>(base + vr[j].unit + CB + v_octet<GS, D>(g * NQ + q, vr[j].row)) = c[j];
          }
        }
      }
    } else {
      const float gl = a.glob[1];
      const Divisor gd = divisor(gl, 0.f);
      const bool whole = s.run && vr[0].unit == vr[1].unit && vr[0].unit == vr[2].unit && vr[0].unit == vr[3].unit;
      const int o = g * NQ + part;
      uint4 mine[4], next[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mine[k] = value(k, o);
        next[k] = value(k, o ^ 1);  // the block's other octet
      }
      uint32_t c[4], sb[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[8], other[8];
        unpack8(mine[k], f);
        unpack8(next[k], other);
        const float amax = fmaxf(amax8(f), amax8(other));
        sb[k] = nvfp4_scale(amax, gd);
        c[k] = nvfp4_octet(f, sb[k], gl, amax);
      }
      if ((o & 1) == 0) {
        const size_t at = 2 * CB + SB + (o >> 1) * 16;
        if (whole) {
          *reinterpret_cast<uint16_t *>(base + vr[0].unit + at + 2 * t) = (uint16_t)(sb[0] | sb[1] << 8);
          *reinterpret_cast<uint16_t *>(base + vr[0].unit + at + 2 * t + 8) = (uint16_t)(sb[2] | sb[3] << 8);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (vr[k].unit >= 0) base[vr[k].unit + at + vr[k].row] = (uint8_t)sb[k];
        }
      }
      if (whole) {
        *reinterpret_cast<uint4 *>(base + vr[0].unit + CB + (part * 32 + lane) * 16) = make_uint4(c[0], c[1], c[2], c[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (vr[k].unit >= 0) *reinterpret_cast<uint32_t *>(base + vr[k].unit + CB + v_octet<GS, D>(o, vr[k].row)) = c[k];
      }
    }
  }
}

// Two codes as fp16 (exact), and an octet's values as bf16 pairs: the product
// with the scale(s) in fp32, then one rounding.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
  return r;
}
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {  // byte I of w
  uint32_t r;
  if constexpr (I == 0) asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(r) : "r"(w));
  if constexpr (I == 1) asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(r) : "r"(w));
  if constexpr (I == 2) asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(r) : "r"(w));
  if constexpr (I == 3) asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, d;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h, float s) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  return bf16x2(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
}
__device__ __forceinline__ uint4 e4m3_values(uint32_t lo, uint32_t hi, float s) {
  return make_uint4(scaled_bf16x2(e4m3x2_to_f16x2(lo), s), scaled_bf16x2(e4m3x2_to_f16x2(lo >> 16), s),
                    scaled_bf16x2(e4m3x2_to_f16x2(hi), s), scaled_bf16x2(e4m3x2_to_f16x2(hi >> 16), s));
}
__device__ __forceinline__ uint4 nvfp4_values(uint32_t w, uint32_t sb, float g) {
  const uint32_t s = __byte_perm(e4m3x2_to_f16x2(sb), 0, 0x1010);  // code times block scale is exact in fp16
  return make_uint4(scaled_bf16x2(hmul2(e2m1x2_to_f16x2<0>(w), s), g), scaled_bf16x2(hmul2(e2m1x2_to_f16x2<1>(w), s), g),
                    scaled_bf16x2(hmul2(e2m1x2_to_f16x2<2>(w), s), g), scaled_bf16x2(hmul2(e2m1x2_to_f16x2<3>(w), s), g));
}

// Bound by HBM: 32048 tokens x 8 heads x 128, E4M3: 197 MB in 34.8 us (5.7 TB/s
// of the measured 6.55); octet by octet, with a sector for every 8 bytes: 52.
template <int FMT, int D>
__global__ void __launch_bounds__(KV_THREADS, 6) kv_read_kernel(KvArgs a, KvRows w) {
  constexpr int NB = D / 32, NQ = D / 64, CB = kv_code_bytes(FMT, D), SB = kv_scale_bytes(FMT, D), GS = kv_granule(FMT);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const long long work = ((long long)w.T + 15) / 16 * a.H * 2, step = (long long)gridDim.x * (KV_THREADS / 32);
  for (long long it = blockIdx.x * (KV_THREADS / 32) + (threadIdx.x >> 5); it < work; it += step) {
    const bool is_v = it & 1;
    if (!(is_v ? w.v_out : w.k_out)) continue;
    const long long ih = it >> 1, grp = ih >> 31 ? ih / a.H : (long long)((uint32_t)ih / (uint32_t)a.H);
    const int h = (int)(ih - grp * a.H);
    const long long t0 = grp * 16;
    const KvGroup s = kv_group<FMT, D>(a, kv_token(w, nullptr, t0), nullptr);
    const uint8_t *base = a.pages + (size_t)h * a.page_units * kv_unit_bytes(FMT, D);
    // granule n of vector i: the octets of the lane's rows, whole or one by one
    if (!is_v) {
      KvRow kr[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) kr[k] = kv_row(s, g + 8 * k);
      const bool whole = s.run && kr[0].unit == kr[1].unit;
      constexpr int NV = NB * 2 * GS / 16;  // vectors
      uint4 x[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (whole) {
          x[i] = *reinterpret_cast<const uint4 *>(base + kr[0].unit + (i * 32 + lane) * 16);
        } else {
          uint32_t *p = reinterpret_cast<uint32_t *>(&x[i]);
#pragma unroll
          for (int n = 0; n < 16 / GS; ++n) {
            const int gi = i * (16 / GS) + n, k = gi & 1;
            if (kr[k].unit < 0) continue;
            const uint8_t *from = base + kr[k].unit + k_octet<GS>(4 * (gi >> 1) + t, kr[k].row);
            if constexpr (GS == 16) x[i] = *reinterpret_cast<const uint4 *>(from);
            if constexpr (GS == 8) {
              const uint2 y = *reinterpret_cast<const uint2 *>(from);
              p[2 * n] = y.x;
              p[2 * n + 1] = y.y;
            }
            if constexpr (GS == 4) p[n] = *reinterpret_cast<const uint32_t *>(from);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (kr[k].unit < 0) continue;
        uint16_t *to = w.k_out + (t0 + kr[k].i) * w.ks + (size_t)h * D + 8 * t;
        const uint8_t *sc = base + kr[k].unit + 2 * CB;
        float fs = 1.f;
        if constexpr (FMT == A_FP8) fs = reinterpret_cast<const float *>(sc)[kr[k].row];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint4 v;
          if constexpr (FMT == A_BF16) v = x[2 * b + k];
          if constexpr (FMT == A_FP8) v = k ? e4m3_values(x[b].z, x[b].w, fs) : e4m3_values(x[b].x, x[b].y, fs);
          if constexpr (FMT == A_NVFP4) {
            const uint4 y = x[b >> 1];
            const uint32_t c = (b & 1) ? (k ? y.w : y.z) : (k ? y.y : y.x);
            v = nvfp4_values(c, sc[kr[k].row * (D / 16) + (t >> 1) * NB + b], a.glob[0]);
          }
          *reinterpret_cast<uint4 *>(to + 32 * b) = v;
        }
      }
    }
    if (is_v) {
      KvRow vr[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) vr[k] = kv_row(s, 2 * t + (k & 1) + 8 * (k >> 1));
      bool same[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)  // with the other octets of its vector
        same[k] = s.run && (FMT == A_FP8 ? vr[k].unit == vr[k ^ 1].unit
                                         : vr[0].unit == vr[1].unit && vr[0].unit == vr[2].unit && vr[0].unit == vr[3].unit);
      constexpr int NV = NQ * 4 * GS / 16;
      uint4 x[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        const int k0 = i * (16 / GS) & 3;  // the first octet's row
        if (GS < 16 && same[k0]) {
          x[i] = *reinterpret_cast<const uint4 *>(base + vr[k0].unit + CB + (i * 32 + lane) * 16);
        } else {
          uint32_t *p = reinterpret_cast<uint32_t *>(&x[i]);
#pragma unroll
          for (int n = 0; n < 16 / GS; ++n) {
            const int gi = i * (16 / GS) + n, k = gi & 3;
            if (vr[k].unit < 0) continue;
            const uint8_t *from = base + vr[k].unit + CB + v_octet<GS, D>(g * NQ + (gi >> 2), vr[k].row);
            if constexpr (GS == 16) x[i] = *reinterpret_cast<const uint4 *>(from);
            if constexpr (GS == 8) {
              const uint2 y = *reinterpret_cast<const uint2 *>(from);
              p[2 * n] = y.x;
              p[2 * n + 1] = y.y;
            }
            if constexpr (GS == 4) p[n] = *reinterpret_cast<const uint32_t *>(from);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (vr[k].unit < 0) continue;
        uint16_t *to = w.v_out + (t0 + vr[k].i) * w.vs + (size_t)h * D + g * (D / 8);
        const uint8_t *sc = base + vr[k].unit + 2 * CB + SB;
        float fs = 1.f;
        if constexpr (FMT == A_FP8) fs = reinterpret_cast<const float *>(sc)[vr[k].row];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          uint4 v;
          if constexpr (FMT == A_BF16) v = x[4 * q + k];
          if constexpr (FMT == A_FP8) {
            const uint4 y = x[2 * q + (k >> 1)];
            v = (k & 1) ? e4m3_values(y.z, y.w, fs) : e4m3_values(y.x, y.y, fs);
          }
          if constexpr (FMT == A_NVFP4) {
            const uint32_t c = k == 0 ? x[q].x : k == 1 ? x[q].y : k == 2 ? x[q].z : x[q].w;
            v = nvfp4_values(c, sc[((g * NQ + q) >> 1) * 16 + vr[k].row], a.glob[1]);
          }
          *reinterpret_cast<uint4 *>(to + 8 * q) = v;
        }
      }
    }
  }
}

// The activation-format constant of a cache description; false if it is not
// one that is built.
bool kv_format(const hq_kv_desc *d, int *fmt) {
  switch (d->dtype) {
    case HQ_BF16: *fmt = A_BF16; break;
    case HQ_E4M3: *fmt = A_FP8; break;
    case HQ_NVFP4: *fmt = A_NVFP4; break;
    default: return false;
  }
  return d->head_dim == 64 || d->head_dim == 128 || d->head_dim == 192 || d->head_dim == 256;
}

size_t kv_page_bytes(const hq_kv_desc *d, int fmt) {
  return (size_t)d->heads * (d->page_size / 16) * kv_unit_bytes(fmt, d->head_dim);
}

KvArgs kv_args(const hq_kv_desc *d, int fmt, int num_pages, const void *pages, const float *glob) {
  KvArgs a{};
  a.H = d->heads;
  a.page = d->page_size;
  a.page_units = d->page_size / 16;
  a.slots_total = (long long)num_pages * d->page_size;
  a.page_bytes = kv_page_bytes(d, fmt);
  a.pages = (uint8_t *)const_cast<void *>(pages);
  a.glob = glob;
  return a;
}

template <class F>
static hq_status kv_dispatch(int fmt, int D, F &&f) {
#define HQ_KV_CASE(FM, DD) \
  if (fmt == FM && D == DD) return f(std::integral_constant<int, FM>{}, std::integral_constant<int, DD>{});
#define HQ_KV_DIMS(FM) HQ_KV_CASE(FM, 64) HQ_KV_CASE(FM, 128) HQ_KV_CASE(FM, 192) HQ_KV_CASE(FM, 256)
  HQ_KV_DIMS(A_BF16)
  HQ_KV_DIMS(A_FP8)
  HQ_KV_DIMS(A_NVFP4)
#undef HQ_KV_DIMS
#undef HQ_KV_CASE
  return HQ_ERR_UNSUPPORTED;
}

static long long kv_blocks(long long warps) { return (warps + KV_THREADS / 32 - 1) / (KV_THREADS / 32); }

hq_status launch_kv_write(int fmt, int D, const KvArgs &a, const KvRows &w, const RopeArgs &rope, cudaStream_t st) {
  return kv_dispatch(fmt, D, [&](auto F, auto DD) {
    const long long kb = kv_blocks(((long long)w.T + 15) / 16 * a.H * 2 * kv_parts(F, DD));
    if (rope.rot) {
      const long long qb = rope.H ? rope_blocks(rope) : 0;
      kv_write_kernel<F, DD, true><<<(unsigned)(kb + qb), KV_THREADS, 0, st>>>(a, w, rope, (unsigned)kb);
    } else {
      kv_write_kernel<F, DD, false><<<(unsigned)kb, KV_THREADS, 0, st>>>(a, w, rope, (unsigned)kb);
    }
    return check_launch();
  });
}

hq_status launch_kv_read(int fmt, int D, const KvArgs &a, const KvRows &w, cudaStream_t st) {
  return kv_dispatch(fmt, D, [&](auto F, auto DD) {
    const long long kb = kv_blocks(((long long)w.T + 15) / 16 * a.H * 2);
    kv_read_kernel<F, DD><<<(unsigned)(kb < 148 * 6 ? kb : 148 * 6), KV_THREADS, 0, st>>>(a, w);
    return check_launch();
  });
}

}  // namespace hq
