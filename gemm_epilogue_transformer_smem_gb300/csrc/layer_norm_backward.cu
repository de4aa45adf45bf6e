// layer_norm_backward.cu -- the kernels of layer norm's backward pass (compiled
// apart from the forward ones to keep builds parallel).
#include "layer_norm_backward.cuh"
#include "layer_norm_kernels.h"

namespace ge_norm {

namespace {

template <class T, bool DROP, bool ADD, int K, bool WIDE>
Kernel held_backward() {
  constexpr int TENSORS = ADD ? 3 : 2, DEPTH = ge::LN_BACKWARD_DEPTH<T>;
  using Ring = std::conditional_t<WIDE, ge::RowRing<T, K, TENSORS, DEPTH>, ge::WordRing<T, K, TENSORS, DEPTH>>;
  return {ge::layer_norm_backward_kernel<T, DROP, ADD, K, WIDE>, ge::HELD_WARP_BYTES<Ring, WIDE>};
}

template <class T, bool DROP, bool ADD>
Kernel held_backward(int k, bool wide) {
  if (!wide) return k == 2 ? held_backward<T, DROP, ADD, 2, false>() : held_backward<T, DROP, ADD, 4, false>();
  return k == 1   ? held_backward<T, DROP, ADD, 1, true>()
         : k == 2 ? held_backward<T, DROP, ADD, 2, true>()
                  : held_backward<T, DROP, ADD, 4, true>();
}

template <class T, bool DROP>
Kernel of(const Shape& s, const Choice& c) {
  if (s.form == NARROW)
    return {c.wide ? ge::layer_norm_backward_narrow_kernel<T, DROP, true> : ge::layer_norm_backward_narrow_kernel<T, DROP, false>,
            ge::NarrowRows<T, ge::LN_NARROW_BACKWARD_ROWS<T>, 3>::WARP_BYTES};
  if (s.form == LONG)
    return {c.wide ? ge::layer_norm_backward_long_kernel<T, DROP, true> : ge::layer_norm_backward_long_kernel<T, DROP, false>, 0};
  return c.add ? held_backward<T, DROP, true>(s.k, c.wide) : held_backward<T, DROP, false>(s.k, c.wide);
}

}  // namespace

Kernel backward_kernel(const Shape& s, const Choice& c) {
  if (c.f32) return c.drop ? of<float, true>(s, c) : of<float, false>(s, c);
  return c.drop ? of<uint16_t, true>(s, c) : of<uint16_t, false>(s, c);
}

void (*const weight_grad_kernel)(const float*, int, int, int, int, float*, float*) = ge::layer_norm_weight_grad_kernel;

}  // namespace ge_norm
