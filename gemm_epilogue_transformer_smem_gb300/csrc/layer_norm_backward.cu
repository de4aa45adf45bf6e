// layer_norm_backward.cu -- the kernels of layer norm's backward pass (compiled
// apart from the forward ones to keep builds parallel).
#include "layer_norm_backward.cuh"
#include "layer_norm_kernels.h"

namespace ge_norm {

namespace {

template <class T, bool DROP, bool ADD, bool WIDE, int... Ks>
Kernel held_backward(int k) {
  Kernel r{nullptr, 0};
  ((k == Ks ? void(r = {ge::layer_norm_backward_kernel<T, DROP, ADD, Ks, WIDE>,
                        ge::RowRing<T, Ks, ADD ? 3 : 2, ge::LN_BACKWARD_DEPTH<T>>::WARP_BYTES})
            : void()), ...);
  return r;
}

template <class T, bool DROP>
Kernel of(const Shape& s, const Choice& c) {
  if (s.form == NARROW)
    return {c.wide ? ge::layer_norm_backward_narrow_kernel<T, DROP, true> : ge::layer_norm_backward_narrow_kernel<T, DROP, false>,
            ge::NarrowRows<T, ge::LN_NARROW_BACKWARD_ROWS<T>, 3>::WARP_BYTES};
  if (s.form == LONG)
    return {c.wide ? ge::layer_norm_backward_long_kernel<T, DROP, true> : ge::layer_norm_backward_long_kernel<T, DROP, false>, 0};
  if (c.add) return c.wide ? held_backward<T, DROP, true, true, 1, 2, 4>(s.k) : held_backward<T, DROP, true, false, 4>(s.k);
  return c.wide ? held_backward<T, DROP, false, true, 1, 2, 4>(s.k) : held_backward<T, DROP, false, false, 4>(s.k);
}

}  // namespace

Kernel backward_kernel(const Shape& s, const Choice& c) {
  if (c.f32) return c.drop ? of<float, true>(s, c) : of<float, false>(s, c);
  return c.drop ? of<uint16_t, true>(s, c) : of<uint16_t, false>(s, c);
}

void (*const weight_grad_kernel)(const float*, int, int, int, int, float*, float*) = ge::layer_norm_weight_grad_kernel;

}  // namespace ge_norm
