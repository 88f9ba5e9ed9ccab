// Attention of one new token per sequence over the paged key-value cache.
#include <cuda_bf16.h>

#include "hq_internal.cuh"

namespace hq {

struct AttnArgs {
  KvArgs kv;
  int B, q_heads, group;       // query heads per kv head
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
};

// The tokens a sequence's query sees: [first, len).
__device__ __forceinline__ int attn_range(const AttnArgs &a, int b, int &first) {
  int n = a.lengths[b];
  const long long most = (long long)a.max_pages * a.kv.page;
  if (n < 0 || n > most) {
    set_device_error(HQ_ERR_DEVICE_INDEX);
    n = n < 0 ? 0 : (int)most;
  }
  first = a.window > 0 && n > a.window ? n - a.window : 0;
  return n;
}

// One CTA per (sequence, query head): 128 tokens at a time, one score per
// thread, then the channels summed over the 128 weights.
template <int FMT, int D>
__global__ void __launch_bounds__(128) attn_kernel(AttnArgs a) {
  __shared__ float sq[D], sp[128], red[4];
  __shared__ const uint8_t *su[128];
  const int b = blockIdx.x / a.q_heads, hq = blockIdx.x % a.q_heads, h = hq / a.group, tid = threadIdx.x;
  int first;
  const int n = attn_range(a, b, first);
  for (int d = tid; d < D; d += 128) sq[d] = bf16_at(a.q + b * a.qs + (size_t)hq * D + d) * a.scale;
  float m = -INFINITY, l = 0.f, acc[(D + 127) / 128];
  for (auto &x : acc) x = 0.f;
  for (int base = first; base < n; base += 128) {
    const int j = base + tid;
    float s = -INFINITY;
    const uint8_t *unit = nullptr;
    int r = 0;
    if (j < n) {
      const int pg = a.page_table[(size_t)b * a.max_pages + j / a.kv.page];
      if (pg < 0 || (long long)pg * a.kv.page >= a.kv.slots_total) {
        set_device_error(HQ_ERR_DEVICE_INDEX);
      } else {
        unit = kv_unit<FMT, D>(a.kv, (long long)pg * a.kv.page + j % a.kv.page, h, r);
      }
    }
    __syncthreads();
    if (unit) {
      s = 0.f;
      for (int o = 0; o < D / 8; ++o) {
        float f[8];
        kv_load<FMT, D>(unit, r, o, false, a.kv.glob, f);
        for (int i = 0; i < 8; ++i) s += f[i] * sq[8 * o + i];
      }
    }
    float mx = s;
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    su[tid] = unit;
    __syncthreads();
    mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float keep = exp2f(m - ref), p = exp2f(s - ref);
    m = mx;
    sp[tid] = p;
    l = l * keep + p;
    __syncthreads();
    for (int c = 0; c * 128 + tid < D; ++c) {
      const int d = c * 128 + tid;
      float x = acc[c] * keep;
      for (int i = 0; i < 128; ++i) {
        if (!su[i]) continue;
        float f[8];
        kv_load<FMT, D>(su[i], (base + i) % 16, d >> 3, true, a.kv.glob, f);
        x += sp[i] * f[d & 7];
      }
      acc[c] = x;
    }
  }
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = l;
  __syncthreads();
  l = red[0] + red[1] + red[2] + red[3];
  for (int c = 0; c * 128 + tid < D; ++c)
    a.out[b * a.os + (size_t)hq * D + c * 128 + tid] = to_bf16(l > 0.f ? acc[c] / l : 0.f);
  if (tid == 0 && a.lse) a.lse[(size_t)b * a.q_heads + hq] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

size_t attn_workspace_bytes(int, int, int, int) { return 256; }

hq_status launch_attn(int fmt, int D, const AttnArgs &a, void *, cudaStream_t st) {
  return kv_dispatch(fmt, D, [&](auto F, auto DD) {
    attn_kernel<F, DD><<<a.B * a.q_heads, 128, 0, st>>>(a);
    return check_launch();
  });
}

}  // namespace hq
