// Host driver for the AdamW step's choice between vectors and single elements (csrc/adamw_access.cuh),
// built and run by tests/test_adamw_access_cpu.py.  Reads lines of
//   state_bits param_dtype grad_dtype param grad master m v
// (addresses as numbers, 0: none) and prints 1 (vectors) or 0 for each.
#include <cstdio>

#include "adamw_access.cuh"

int main() {
  int bits, p, g;
  unsigned long long a[5];
  while (std::scanf("%d %d %d %llu %llu %llu %llu %llu", &bits, &p, &g, a, a + 1, a + 2, a + 3, a + 4) == 8) {
    moe_adamw_tensor t{};
    t.state_bits = bits;
    t.param_dtype = p;
    t.grad_dtype = g;
    t.param = reinterpret_cast<void*>(a[0]);
    t.grad = reinterpret_cast<const void*>(a[1]);
    t.master = reinterpret_cast<float*>(a[2]);
    t.m = reinterpret_cast<void*>(a[3]);
    t.v = reinterpret_cast<void*>(a[4]);
    std::printf("%d\n", moe::adamw_by_vectors(t) ? 1 : 0);
  }
  return 0;
}
