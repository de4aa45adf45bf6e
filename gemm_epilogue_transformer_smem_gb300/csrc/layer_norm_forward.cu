// layer_norm_forward.cu -- the kernels of layer norm's forward pass (compiled
// apart from the backward ones to keep builds parallel).
#include "layer_norm_kernels.h"

namespace ge_norm {

namespace {

template <class T, bool DROP, bool ADD, int K, int R, bool WIDE>
Kernel held_forward() {
  using Ring = std::conditional_t<WIDE, ge::RowRing<T, K, ADD ? 2 : 1, R>, ge::WordRing<T, K, ADD ? 2 : 1, R>>;
  return {ge::layer_norm_kernel<T, DROP, ADD, K, R, WIDE>, ge::HELD_WARP_BYTES<Ring, WIDE>};
}

template <class T, bool DROP, bool ADD>
Kernel held_forward(const Shape& s, bool wide) {
  if (!wide) return s.k == 2 ? held_forward<T, DROP, ADD, 2, 1, false>() : held_forward<T, DROP, ADD, 4, 1, false>();
  if (s.k == 2 && s.rows == 1) return held_forward<T, DROP, ADD, 2, 1, true>();
  if constexpr (sizeof(T) == 2)
    return held_forward<T, DROP, ADD, 4, 2, true>();
  else
    return s.k == 2 ? held_forward<T, DROP, ADD, 2, 2, true>() : held_forward<T, DROP, ADD, 4, 1, true>();
}

template <class T, bool DROP>
Kernel of(const Shape& s, const Choice& c) {
  if (s.form == NARROW)
    return {c.wide ? ge::layer_norm_narrow_kernel<T, DROP, true> : ge::layer_norm_narrow_kernel<T, DROP, false>,
            ge::NarrowRows<T, ge::LN_NARROW_ROWS<T>, 2>::WARP_BYTES};
  if (s.form == LONG)
    return {c.wide ? ge::layer_norm_long_kernel<T, DROP, true> : ge::layer_norm_long_kernel<T, DROP, false>, 0};
  if (DROP || c.add) return held_forward<T, DROP, true>(s, c.wide);  // dropout alone adds zeros
  return held_forward<T, false, false>(s, c.wide);
}

}  // namespace

Kernel forward_kernel(const Shape& s, const Choice& c) {
  if (c.f32) return c.drop ? of<float, true>(s, c) : of<float, false>(s, c);
  return c.drop ? of<uint16_t, true>(s, c) : of<uint16_t, false>(s, c);
}

}  // namespace ge_norm
