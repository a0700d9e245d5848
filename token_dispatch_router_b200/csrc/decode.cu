// Host side of the few-token layer: workspace layout and the launches (router, first
// expert product, second expert product with the sum over experts, partial sums of cut tiles).
#include "few.cuh"
#include "few_args.cuh"

namespace moe {

moe_status launch_few_route(const moe_shape& s, const void* x, const void* w_r, const float* bias,
                            const float* logits_in, int32_t* ids, float* w, uint32_t* clear,
                            int n_clear, cudaStream_t st);
int few_up_pieces();
size_t few_up_part_bytes(int T);
moe_status launch_few_up(FewUpArgs a, int d, int n_experts, const void* x, const void* w_gate,
                         const void* w_up, cudaStream_t st);
size_t few_down_part_bytes(int T);
moe_status launch_few_down(FewDownArgs a, const void* w_down, cudaStream_t st);

namespace {

struct Layout {
  size_t arrived, ids, w, act, part, total;
  int active;  // experts that can have a token
};
Layout layout(const moe_shape& s) {
  Layout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) & ~(size_t)255;
    return at;
  };
  const size_t A = (size_t)s.T * s.K;
  L.active = A < (size_t)s.E ? (int)A : s.E;
  L.arrived = take((size_t)few_up_pieces() * 4);
  L.ids = take(A * 4);
  L.w = take(A * 4);
  L.act = take((size_t)L.active * s.T * s.n * 2);
  // one after the other: few_down's partials may overwrite few_up's
  const size_t up = few_up_part_bytes(s.T), down = few_down_part_bytes(s.T);
  L.part = take(up > down ? up : down);
  L.total = o;
  return L;
}

}  // namespace

size_t decode_workspace_bytes(const moe_shape& s) { return layout(s).total; }

moe_status launch_decode(const moe_shape& s, const void* x, const void* w_r, const float* bias,
                         const float* logits_in, const void* w_gate, const void* w_up,
                         const void* w_down, void* out, int cap, uint8_t* ws, cudaStream_t st) {
  const Layout L = layout(s);
  int32_t* ids = (int32_t*)(ws + L.ids);
  float* w = (float*)(ws + L.w);
  FewUpArgs u = {};
  u.T = s.T;
  u.K = s.K;
  u.E = s.E;
  u.n = s.n;
  u.cap = cap;
  u.ids = ids;
  u.topk_w = w;
  u.act = (bf16*)(ws + L.act);
  u.part = (float*)(ws + L.part);
  u.arrived = (uint32_t*)(ws + L.arrived);
  FewDownArgs dn = {};
  dn.T = s.T;
  dn.K = s.K;
  dn.E = s.E;
  dn.cap = cap;
  dn.n = s.n;
  dn.d = s.d;
  dn.act = u.act;
  dn.rows = L.active * s.T;
  dn.part = u.part;
  dn.ids = ids;
  dn.out = (bf16*)out;
  moe_status r;
  if ((r = launch_few_route(s, x, w_r, bias, logits_in, ids, w, u.arrived,
                            few_up_pieces(), st)) !=
      MOE_OK)
    return r;
  if ((r = launch_few_up(u, s.d, s.E, x, w_gate, w_up, st)) != MOE_OK) return r;
  return launch_few_down(dn, w_down, st);
}

}  // namespace moe
