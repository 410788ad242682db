// Stands in for the runtime's launch call: counts launches and lets the first `good` of them pass, without any device.
extern "C" {
int bllm_test_launches = 0, bllm_test_good = 0;
int hipLaunchKernel(const void*, unsigned long, unsigned, unsigned long, unsigned, void**, unsigned long, void*) {
  return bllm_test_launches++ < bllm_test_good ? 0 : 1;
}
int hipGetLastError() { return 0; }
}
