/* Stand-in for the HIP runtime's allocation calls, preloaded over the library so that its
 * buffers can be followed without a GPU: one device, `limit` bytes of memory, never touched.
 * Prints "alloc ADDRESS BYTES" and "free ADDRESS". */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

static uintptr_t next = 0x100000;

int hipGetDevice(int* dev) { *dev = 0; return 0; }
int hipSetDevice(int dev) { return dev != 0; }
int hipDeviceSynchronize(void) { return 0; }
int hipGetLastError(void) { return 0; }

int hipMalloc(void** p, size_t bytes) {
  if (bytes > (size_t)atoll(getenv("SHIM_LIMIT"))) return 2;
  *p = (void*)next;
  next += (bytes + 0xFFF) / 0x1000 * 0x1000;
  printf("alloc %p %zu\n", *p, bytes);
  fflush(stdout);
  return 0;
}

int hipFree(void* p) {
  printf("free %p\n", p);
  fflush(stdout);
  return 0;
}
