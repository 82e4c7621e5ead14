// Takes the place of the HIP calls that a launch makes and notes them, so that a test can see on a
// machine without a GPU which kernels a call would launch, on which grid and with how much LDS.
#include <stddef.h>
#include <stdint.h>

namespace {
struct Event {
  const void* kernel;
  uint32_t grid[3], block[3];
  int64_t lds;      // of a launch
  int64_t allowed;  // most dynamic LDS, where it is set; -1 for a launch
};
Event events[4096];
int count = 0;
struct Dim3 {
  uint32_t x, y, z;
};
struct {
  Dim3 grid, block;
  size_t lds;
  void* stream;
} pushed;   // <<< >>> of the launch under way
}  // namespace

extern "C" {
int hipFuncSetAttribute(const void* kernel, int, int value) {
  if (count < 4096) events[count++] = {kernel, {0, 0, 0}, {0, 0, 0}, 0, value};
  return 0;
}
int __hipPushCallConfiguration(Dim3 grid, Dim3 block, size_t lds, void* stream) {
  pushed = {grid, block, lds, stream};
  return 0;
}
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* lds, void** stream) {
  *grid = pushed.grid;
  *block = pushed.block;
  *lds = pushed.lds;
  *stream = pushed.stream;
  return 0;
}
int hipLaunchKernel(const void* kernel, Dim3 grid, Dim3 block, void**, size_t lds, void*) {
  if (count < 4096)
    events[count++] = {kernel, {grid.x, grid.y, grid.z}, {block.x, block.y, block.z}, (int64_t)lds, -1};
  return 0;
}
int hipGetLastError() { return 0; }
int recorder_take(Event* out) {
  const int n = count;
  for (int i = 0; i < n; ++i) out[i] = events[i];
  count = 0;
  return n;
}
}
