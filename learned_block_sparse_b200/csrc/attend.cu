// Attention of new tokens: the choice of passes, splits and kernels, the workspace
// layout, and the merge of partial results.
#include "attend_common.cuh"

namespace eta {

namespace {

// One warp per (token, head): the slots' partials, added in slot order with the
// weights 2^(m_s - max m); bytes: slots x (D + 2) x 4 read per row.
template <int D>
__global__ void __launch_bounds__(256) attend_merge_kernel(const AttendArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t rows = a.T * a.Hq;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows || !token_live(a, row / a.Hq)) return;
  const int slots = a.own_splits + (a.P > 0 ? a.prefix_splits : 0);
  float M = -INFINITY;
  for (int s = lane; s < slots; s += 32) M = fmaxf(M, a.ml_part[s * rows + row].x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  constexpr int V = D / 32;
  float o[V], L = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
  for (int s = 0; s < slots; ++s) {
    const float2 ml = a.ml_part[s * rows + row];
    if (!(ml.y > 0.0f)) continue;  // a range without a visible key
    const float c = exp2f(ml.x - M);
    L = fmaf(c, ml.y, L);
    const float* p = a.o_part + (s * rows + row) * D + lane;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(c, p[32 * i], o[i]);
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) store_out(a.out, a.out_dtype, row * D + lane + 32 * i, o[i] * inv);
}

constexpr int kSimtRows = 16;

// Splits of a pass of `items` tiles so that about `want` thread blocks run.
int splits_for(int64_t items, int64_t want, int64_t key_tiles) {
  int64_t s = (want + items - 1) / items;
  if (s > key_tiles) s = key_tiles;
  if (s > 128) s = 128;
  return static_cast<int>(s < 1 ? 1 : s);
}

struct Plan {
  int own, prefix;  // splits
};

Plan plan_of(const eta_shape_t& s, int64_t T, bool single, int64_t own_keys, int64_t P) {
  const int G = s.n_q_heads / s.n_kv_heads;
  const int64_t qt = kSimtRows / G, want = 4 * static_cast<int64_t>(device_sm_count());
  Plan p;
  const int64_t own_items = single ? s.batch : (T + qt - 1) / qt;
  p.own = splits_for(own_items * s.n_kv_heads, want, (own_keys + 31) / 32);
  p.prefix = P > 0 ? splits_for((T + qt - 1) / qt * s.n_kv_heads, want, (P + 31) / 32) : 0;
  return p;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Partial rows (slots x rows) a pass of tiles of R rows can leave for up to T
// queries: splits <= want / items + 1 and rows <= R x items, so at most
// R (want + items); without a second pass a pass of `want` tiles or more is never
// split and leaves none. Non-decreasing in T.
static int64_t partial_rows(int64_t items, int64_t R, int64_t want, bool second) {
  if (!second && items > want) items = want;
  return R * (want + items);
}

size_t attend_workspace_bytes(const eta_shape_t& s, int64_t T, bool with_prefix) {
  const int64_t G = s.n_q_heads / s.n_kv_heads, qt = kSimtRows / G, want = 4 * static_cast<int64_t>(device_sm_count());
  const int64_t tiles = (T + qt - 1) / qt * s.n_kv_heads;
  int64_t rows = partial_rows(tiles, kSimtRows, want, with_prefix);
  const int64_t single = partial_rows(T * s.n_kv_heads, G, want, with_prefix);  // one query per row and tile
  if (single > rows) rows = single;
  if (with_prefix) rows += partial_rows(tiles, kSimtRows, want, true);
  return kWsHeaderBytes + align256(static_cast<size_t>(rows) * sizeof(float2)) +
         align256(static_cast<size_t>(rows) * s.head_dim * sizeof(float));
}

cudaError_t launch_attend(const AttendCall& c, cudaStream_t st) {
  AttendArgs a = make_attend_args(c);
  const int D = c.shape.head_dim;
  const int64_t own_keys = a.sinks + a.window < a.n ? a.sinks + a.window : a.n;
  const Plan p = plan_of(c.shape, a.T, a.cu_q == nullptr, own_keys, a.P);
  a.own_splits = p.own;
  a.prefix_splits = p.prefix;
  const int slots = p.own + p.prefix;
  if (slots > 1) {
    unsigned char* w = static_cast<unsigned char*>(c.ws) + kWsHeaderBytes;
    const size_t rows = static_cast<size_t>(a.T) * a.Hq;
    a.ml_part = reinterpret_cast<float2*>(w);
    a.o_part = reinterpret_cast<float*>(w + align256(slots * rows * sizeof(float2)));
  }
  cudaError_t e = cudaSuccess;
  if (a.P > 0) e = launch_attend_simt(a, c.shape.kv_dtype, D, true, st);
  if (e == cudaSuccess) e = launch_attend_simt(a, c.shape.kv_dtype, D, false, st);
  if (e != cudaSuccess || slots == 1) return e;
  return D == 128 ? launch_pdl(attend_merge_kernel<128>, static_cast<unsigned>((a.T * a.Hq + 7) / 8), 256u, 0, st, a)
                  : launch_pdl(attend_merge_kernel<64>, static_cast<unsigned>((a.T * a.Hq + 7) / 8), 256u, 0, st, a);
}

}  // namespace eta
