/* Stands in for the HIP runtime where there is no GPU: writes down what a library launches
 * (and the attributes that it sets) instead of doing it. Loaded ahead of the library
 * with its symbols global. rec_log() returns lines of
 *   launch <device> <kernel> <workgroups> <threads> <dynamic LDS>
 *   attribute <device> <kernel> <value>
 * since the last rec_start(device, failures): the current device, and how many of the
 * next attribute calls are to fail. */
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

typedef struct { uint32_t x, y, z; } dim3;
typedef struct { dim3 grid, block; size_t lds; void* stream; } config;
enum { kMost = 4096 };
static const void* functions[kMost];
static const char* names[kMost];
static int count, device, failures;
static config pushed[16];
static int depth;
static char text[1 << 16];

static const char* name_of(const void* f) {
  for (int i = 0; i < count; ++i)
    if (functions[i] == f) return names[i];
  return "?";
}
static void append(const char* line) { strncat(text, line, sizeof text - strlen(text) - 1); }

void rec_start(int dev, int fail) { device = dev, failures = fail, text[0] = 0; }
const char* rec_log(void) { return text; }
int rec_kernels(void) { return count; }
const char* rec_kernel(int i) { return names[i]; }

void** __hipRegisterFatBinary(const void* data) {
  static void* handle;
  (void)data;
  return &handle;
}
void __hipUnregisterFatBinary(void** handle) { (void)handle; }
void __hipRegisterFunction(void** modules, const void* host, char* dev, const char* name, unsigned limit, void* tid,
                           void* bid, dim3* block, dim3* grid, int* size) {
  (void)modules, (void)dev, (void)limit, (void)tid, (void)bid, (void)block, (void)grid, (void)size;
  if (count < kMost) functions[count] = host, names[count++] = name;
}
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void* stream) {
  pushed[depth++] = (config){grid, block, lds, stream};
  return 0;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, void** stream) {
  const config c = pushed[--depth];
  *grid = c.grid, *block = c.block, *lds = c.lds, *stream = c.stream;
  return 0;
}
int hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds, void* stream) {
  char line[1024];
  (void)args, (void)stream;
  snprintf(line, sizeof line, "launch %d %s %llu %u %zu\n", device, name_of(f),
           (unsigned long long)grid.x * grid.y * grid.z, block.x * block.y * block.z, lds);
  append(line);
  return 0;
}
int hipFuncSetAttribute(const void* f, int attribute, int value) {
  char line[1024];
  (void)attribute;
  if (failures > 0) {
    --failures;
    return 1;
  }
  snprintf(line, sizeof line, "attribute %d %s %d\n", device, name_of(f), value);
  append(line);
  return 0;
}
int hipGetDevice(int* d) {
  *d = device;
  return 0;
}
int hipGetLastError(void) { return 0; }
