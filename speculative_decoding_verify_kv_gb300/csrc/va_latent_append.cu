// Rows into a latent cache: the latent part normalised, the shared key part
// and the queries' rope parts rotated, each written to its place.
//
// Per row: c = x / sqrt(mean(x^2) + eps) * w over latent_dim values, and for
// each of the 32 pairs (a, b) of a rope part (a cos - b sin, a sin + b cos).
// Bound by bytes: every value is read and written once, 16 bytes at a time,
// and a row's angles are loaded once for all the heads that a thread turns.
// One CTA per row (one warp for the cache row, four for the queries), so that
// neither waits for the other.
#include <string.h>

#include "va_common.cuh"
#include "va_host.h"

namespace va {

constexpr int kRope = 64;
constexpr int kQueryThreads = 128;
constexpr int kAppendThreads = kQueryThreads + 32;

struct AppendParams {
  int rows, heads, positions, interleaved;
  float eps;
  const void* kv;
  long long kv_stride;
  const void* weight;
  const float* rope;
  const int* position;
  const long long* slot;
  long long slots;
  const void* q_rope;
  long long q_row, q_head;
  void* q;
  void* cache;
  unsigned* status;
};

// 16 bytes of elements as fp32.  VEC: the address is a multiple of 16 bytes.
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const T* at, float (&x)[16 / sizeof(T)]) {
  constexpr int E = 16 / sizeof(T);
  T raw[E];
  if (VEC) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    memcpy(raw, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) raw[i] = at[i];
  }
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = (float)raw[i];
}

template <typename T>
__device__ __forceinline__ void store16(T* at, const float (&x)[16 / sizeof(T)]) {
  constexpr int E = 16 / sizeof(T);
  T raw[E];
#pragma unroll
  for (int i = 0; i < E; ++i) raw[i] = T(x[i]);
  uint4 v;
  memcpy(&v, raw, 16);
  *reinterpret_cast<uint4*>(at) = v;
}

// A thread's share of a rope part: pairs E c .. E c + E - 1, two pieces of 16
// bytes, at elements first(c) and second(c).
template <typename T>
struct Turn {
  static constexpr int E = 16 / sizeof(T);
  static constexpr int LANES = kRope / 2 / E;  // threads to a rope part
  float cs[E], sn[E];
  int first, second;
  bool inter;
  __device__ __forceinline__ Turn(const float* angles, int c, bool interleaved) : inter(interleaved) {
    first = interleaved ? 2 * E * c : E * c;
    second = interleaved ? first + E : first + kRope / 2;
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(angles + E * c + i);
      const float4 b = *reinterpret_cast<const float4*>(angles + kRope / 2 + E * c + i);
      cs[i] = a.x, cs[i + 1] = a.y, cs[i + 2] = a.z, cs[i + 3] = a.w;
      sn[i] = b.x, sn[i + 1] = b.y, sn[i + 2] = b.z, sn[i + 3] = b.w;
    }
  }
  __device__ __forceinline__ void apply(float (&x)[E], float (&y)[E]) const {
    if (inter) {  // pair i is values 2i and 2i + 1 of the two pieces laid end to end
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * cs[i] - b * sn[i];
        x[2 * i + 1] = a * sn[i] + b * cs[i];
        const float c = y[2 * i], d = y[2 * i + 1];
        y[2 * i] = c * cs[E / 2 + i] - d * sn[E / 2 + i];
        y[2 * i + 1] = c * sn[E / 2 + i] + d * cs[E / 2 + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float a = x[i], b = y[i];
        x[i] = a * cs[i] - b * sn[i];
        y[i] = a * sn[i] + b * cs[i];
      }
    }
  }
};

template <typename T, int LATENT, bool VEC>
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(const AppendParams p) {
  constexpr int E = 16 / sizeof(T);
  constexpr int WIDTH = LATENT + kRope;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int r = blockIdx.x, tid = threadIdx.x;
  const int pos = p.position[r];
  if (pos == -1) return;
  if (pos < 0 || pos >= p.positions) {
    if (tid == 0) flag(p.status, VA_DEV_CTX_OVERFLOW);
    return;
  }
  const long long slot = p.slot[r];
  if (slot < -1 || slot >= p.slots) {
    if (tid == 0) flag(p.status, VA_DEV_BAD_BLOCK);
    return;
  }
  const float* angles = p.rope + (long long)pos * kRope;
  if (tid < kQueryThreads) {
    // One head at a time: with two or four of them under way a thread's registers
    // cost more CTAs than its loads gain (4,096 rows of 128 heads: 28 us, 34, 45).
    constexpr int L = Turn<T>::LANES;
    if (tid / L >= p.heads) return;
    const Turn<T> turn(angles, tid % L, p.interleaved != 0);
    const T* from = reinterpret_cast<const T*>(p.q_rope) + r * p.q_row;
    T* to = reinterpret_cast<T*>(p.q) + (long long)r * p.heads * WIDTH + LATENT;
#pragma unroll 1
    for (int h = tid / L; h < p.heads; h += kQueryThreads / L) {
      float x[E], y[E];
      load16<T, VEC>(from + h * p.q_head + turn.first, x);
      load16<T, VEC>(from + h * p.q_head + turn.second, y);
      turn.apply(x, y);
      store16<T>(to + (long long)h * WIDTH + turn.first, x);
      store16<T>(to + (long long)h * WIDTH + turn.second, y);
    }
    return;
  }
  if (slot < 0) return;
  const int lane = tid & 31;
  constexpr int PIECES = LATENT / E / 32;
  const T* row = reinterpret_cast<const T*>(p.kv) + r * p.kv_stride;
  T* out = reinterpret_cast<T*>(p.cache) + slot * WIDTH;
  float x[PIECES][E], w[PIECES][E];
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < PIECES; ++k) load16<T, VEC>(row + (lane + 32 * k) * E, x[k]);
  if (lane < Turn<T>::LANES) {
    const Turn<T> turn(angles, lane, p.interleaved != 0);
    float a[E], b[E];
    load16<T, VEC>(row + LATENT + turn.first, a);
    load16<T, VEC>(row + LATENT + turn.second, b);
    turn.apply(a, b);
    store16<T>(out + LATENT + turn.first, a);
    store16<T>(out + LATENT + turn.second, b);
  }
  if (p.weight) {
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      load16<T, VEC>(reinterpret_cast<const T*>(p.weight) + (lane + 32 * k) * E, w[k]);
#pragma unroll
      for (int i = 0; i < E; ++i) sum = fmaf(x[k][i], x[k][i], sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float f = 1.f / sqrtf(sum / LATENT + p.eps);
#pragma unroll
    for (int k = 0; k < PIECES; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) x[k][i] *= f * w[k][i];
  }
#pragma unroll
  for (int k = 0; k < PIECES; ++k) store16<T>(out + (lane + 32 * k) * E, x[k]);
}

template <typename T, int LATENT>
static cudaError_t launch_append(const AppendParams& q, bool vec, cudaStream_t st) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)q.rows);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(
      &cfg, vec ? latent_append_kernel<T, LATENT, true> : latent_append_kernel<T, LATENT, false>, q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace va

using namespace va;

extern "C" {

va_status verify_attn_latent_append(const va_latent* kv, const va_latent_rows* n, uint32_t* status, void* stream) {
  if (!kv || !n || n->num_rows < 0 || n->num_heads < 0) return VA_ERR_INVALID_ARG;
  if (kv->dtype < VA_F32 || kv->dtype > VA_Q8_0) return VA_ERR_INVALID_ARG;
  if (kv->dtype == VA_Q8_0) return VA_ERR_UNSUPPORTED;
  if ((kv->latent_dim != 256 && kv->latent_dim != 512) || kv->rope_dim != kRope) return VA_ERR_UNSUPPORTED;
  if (n->num_heads > VA_MAX_LATENT_HEADS) return VA_ERR_UNSUPPORTED;
  if (!(n->norm_eps >= 0.f) || n->rope_positions < 1 || n->num_slots < 1) return VA_ERR_INVALID_ARG;
  if (n->interleaved != 0 && n->interleaved != 1) return VA_ERR_INVALID_ARG;
  const int width = kv->latent_dim + kv->rope_dim;
  if (n->num_rows > 1 && n->kv_stride < width) return VA_ERR_INVALID_ARG;
  if (n->num_rows > 0 && (!kv->cache || !n->kv || !n->rope || !n->position || !n->slot)) return VA_ERR_INVALID_ARG;
  if (n->num_rows > 0 && n->num_heads > 0) {
    if (!n->q_rope || !n->q) return VA_ERR_INVALID_ARG;
    if ((n->num_heads > 1 && n->q_head_stride < kRope) || (n->num_rows > 1 && n->q_row_stride < kRope))
      return VA_ERR_INVALID_ARG;
  }
  const int size = kv->dtype == VA_F32 ? 4 : 2;
  const uintptr_t from = (uintptr_t)n->kv | (uintptr_t)n->norm_weight | (uintptr_t)n->q_rope;
  if (((uintptr_t)kv->cache | (uintptr_t)n->q | (uintptr_t)n->rope) % 16 || from % size || (uintptr_t)n->slot % 8)
    return VA_ERR_ALIGNMENT;
  if (n->num_rows == 0) return VA_OK;
  cudaStream_t cs = (cudaStream_t)stream;
  va_status st = check_stream_device(cs);
  if (st != VA_OK) return st;
  AppendParams q;
  memset(&q, 0, sizeof(q));
  q.rows = n->num_rows;
  q.heads = n->num_heads;
  q.positions = n->rope_positions;
  q.interleaved = n->interleaved;
  q.eps = n->norm_eps;
  q.kv = n->kv;
  q.kv_stride = n->kv_stride;
  q.weight = n->norm_weight;
  q.rope = n->rope;
  q.position = n->position;
  q.slot = (const long long*)n->slot;
  q.slots = n->num_slots;
  q.q_rope = n->q_rope;
  q.q_row = n->q_row_stride;
  q.q_head = n->q_head_stride;
  q.q = n->q;
  q.cache = kv->cache;
  q.status = (unsigned*)status;
  // 16-byte loads where every piece that is read starts on a multiple of 16
  // bytes, else element by element.
  const bool vec = from % 16 == 0 && n->kv_stride * size % 16 == 0 &&
                   (n->num_heads == 0 || (n->q_row_stride * size % 16 == 0 && n->q_head_stride * size % 16 == 0));
  cudaError_t e;
  if (kv->dtype == VA_F32)
    e = kv->latent_dim == 512 ? launch_append<float, 512>(q, vec, cs) : launch_append<float, 256>(q, vec, cs);
  else
    e = kv->latent_dim == 512 ? launch_append<__nv_bfloat16, 512>(q, vec, cs)
                              : launch_append<__nv_bfloat16, 256>(q, vec, cs);
  return e == cudaSuccess ? VA_OK : note_cuda(e);
}

}  // extern "C"
