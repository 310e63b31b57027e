// Attention over the quantized KV cache, the plain way: a block per (sequence, new token, query head), a warp per slot, fp32.
#include "kv_common.cuh"

namespace pace {
namespace kv {

template <int D, int BITS, int IO32>
__global__ void __launch_bounds__(128) attend_simple(KvDev c, KvTensor q, const uint32_t *__restrict__ mask, float scale,
                                                     KvTensor o) {
  using L = Tile<D, BITS>;
  constexpr int E = D / 32;      // elements a lane: dims lane*E ..
  const int h = blockIdx.x % c.Hq, t = (blockIdx.x / c.Hq) % c.n_tokens, b = blockIdx.x / c.Hq / c.n_tokens;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, kvh = h / c.group;
  const long len = max(c.lens[b], 0);
  const int n = new_tokens(c, b), words = (c.n_tokens + 31) / 32;
  float acc[E] = {}, m = -INFINITY, l = 0.0f, qv[E];
  for (int i = 0; i < E; ++i) qv[i] = load_io(q.p, b * q.sb + t * q.st + h * q.sh + lane * E + i, c.io) * scale;
  const long total = t < n ? len + n : 0;
  for (long slot = w; slot < total; slot += 4) {
    if (slot >= len) {
      const int j = (int)(slot - len);
      if (!(mask ? (mask[((long)b * c.n_tokens + t) * words + j / 32] >> (j & 31)) & 1 : j <= t)) continue;
    }
    const int page = page_of(c, b, slot);
    if (page < 0) {
      if (lane == 0) atomicOr(c.status, PACE_KV_BAD_PAGE);
      continue;
    }
    const char *tile = tile_at<L::BYTES>(c, page, kvh, slot);
    const int tt = (int)(slot % TILE), a = lane * E / 8, p = (a >> 3) * TILE + L::pos(tt);
    float kv[2][E];
    for (int part = 0; part < 2; ++part) {
      const char *at = tile + (part ? L::v8(tt, a) : L::k8(tt, a));
      uint2 wd = make_uint2(reinterpret_cast<const uint32_t *>(at)[0], BITS == 8 ? reinterpret_cast<const uint32_t *>(at)[1] : 0);
      int u[8];
      unpack8<BITS>(wd, u);
      const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(tile + (part ? L::VS : L::KS))[p]);
      const int z = BITS == 4 ? reinterpret_cast<const uint8_t *>(tile + (part ? L::VZ : L::KZ))[p] : 128;
      for (int i = 0; i < E; ++i) {
        int ui = 0;
        for (int e = 0; e < 8; ++e) ui = (lane * E + i) % 8 == e ? u[e] : ui;
        kv[part][i] = s * (float)(ui - z);
      }
    }
    float d = 0.0f;
    for (int i = 0; i < E; ++i) d += qv[i] * kv[0][i];
    d = warp_sum(d);
    const float mn = fmaxf(m, d), al = expf(m - mn), pr = expf(d - mn);
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * al + pr * kv[1][i];
    l = l * al + pr;
    m = mn;
  }
  __shared__ float sm[4], sl[4], sa[4][D];
  if (lane == 0) sm[w] = m, sl[w] = l;
  for (int i = 0; i < E; ++i) sa[w][lane * E + i] = acc[i];
  __syncthreads();
  const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  for (int e = threadIdx.x; e < D; e += 128) {
    float s = 0.0f, lt = 0.0f;
    for (int i = 0; i < 4; ++i) {
      const float f = sm[i] == -INFINITY ? 0.0f : expf(sm[i] - mm);
      s += f * sa[i][e];
      lt += f * sl[i];
    }
    store_io(o.p, b * o.sb + t * o.st + h * o.sh + e, lt > 0.0f ? s / lt : 0.0f, c.io);
  }
}

}  // namespace kv
}  // namespace pace

namespace {
template <int D, int BITS>
cudaError_t go(const KvDev &c, const KvTensor &q, const uint32_t *mask, float scale, const KvTensor &o, cudaStream_t s) {
  const unsigned blocks = (unsigned)c.batch * c.n_tokens * c.Hq;
  pace::kv::attend_simple<D, BITS, 0><<<blocks, 128, 0, s>>>(c, q, mask, scale, o);
  return cudaGetLastError();
}
}  // namespace

void pace_kv_attend_work(const pace_kv_config &, size_t *count_bytes, size_t *part_bytes) {
  *count_bytes = 256;
  *part_bytes = 256;
}

cudaError_t pace_launch_kv_attend(const KvDev &c, const KvTensor &q, const uint32_t *mask, float scale, const KvTensor &o,
                                  cudaStream_t s) {
  if (c.bits == 4) return c.d == 64 ? go<64, 4>(c, q, mask, scale, o, s) : c.d == 128 ? go<128, 4>(c, q, mask, scale, o, s) : go<256, 4>(c, q, mask, scale, o, s);
  return c.d == 64 ? go<64, 8>(c, q, mask, scale, o, s) : c.d == 128 ? go<128, 8>(c, q, mask, scale, o, s) : go<256, 8>(c, q, mask, scale, o, s);
}
