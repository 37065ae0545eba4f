// The attention calls on a machine without a GPU, as launch_probe.cpp makes other
// calls: its stand-ins for the HIP runtime record every launch and refuse what HIP
// refuses.  Pointers are numbers that nobody follows.
//   attn_launch_probe library call T B heads kv_heads D page
#define main launch_probe_main
#include "launch_probe.cpp"
#undef main

#include "../include/ufp4.h"

template <class F>
static F get(void* lib, const char* name) {
  return (F)dlsym(lib, name);
}

int main(int argc, char** argv) {
  void* lib = argc == 9 ? dlopen(argv[1], RTLD_NOW) : nullptr;
  if (!lib) {
    fprintf(stderr, "%s\n", dlerror());
    return 2;
  }
  const std::string call = argv[2];
  const int64_t T = atoll(argv[3]);
  const int32_t B = atoi(argv[4]), H = atoi(argv[5]), K = atoi(argv[6]), D = atoi(argv[7]);
  auto at = [](int64_t i) { return (void*)(i << 44); };
  const int32_t* starts = (const int32_t*)at(20);
  const int64_t ldq = (int64_t)H * D, ldk = (int64_t)K * D;
  ufp4_kv_cache c = {};
  c.k_codes = (uint8_t*)at(21);
  c.k_scales = at(22);
  c.v_codes = (uint8_t*)at(23);
  c.v_scales = at(24);
  c.pages = 1000;
  c.page_tokens = atoi(argv[8]);
  c.kv_heads = K;
  c.D = D;
  c.cfg.grid = UFP4_INT4;
  c.cfg.block_rows = 1;
  c.cfg.block_cols = 16;
  c.cfg.rht_n = 16;
  const int32_t* lens = (const int32_t*)at(25);
  const int32_t* table = (const int32_t*)at(26);
  int st = -100;
  if (call == "attn_fwd")
    st = get<decltype(&ufp4_attn_fwd)>(lib, "ufp4_attn_fwd")(at(1), ldq, at(2), ldk, at(3), ldk, starts, B, T, H, K, D, 0.1f, at(4), ldq,
                                                            (float*)at(5), nullptr);
  else if (call == "attn_bwd")
    st = get<decltype(&ufp4_attn_bwd)>(lib, "ufp4_attn_bwd")(at(1), ldq, at(2), ldk, at(3), ldk, starts, B, T, H, K, D, 0.1f, at(4), ldq,
                                                            (const float*)at(5), at(6), ldq, at(7), ldq, at(8), ldk, at(9), ldk, at(10),
                                                            (size_t)1 << 43, nullptr);
  else if (call == "kv_write")
    st = get<decltype(&ufp4_kv_write)>(lib, "ufp4_kv_write")(at(1), ldk, at(2), ldk, starts, B, T, lens, table, 8, 8, &c, nullptr);
  else if (call == "kv_read")
    st = get<decltype(&ufp4_kv_read)>(lib, "ufp4_kv_read")(&c, starts, B, T, lens, table, 8, 8, at(1), ldk, at(2), ldk, nullptr);
  else if (call == "kv_attn")
    st = get<decltype(&ufp4_kv_attn)>(lib, "ufp4_kv_attn")(at(1), ldq, starts, B, T, H, lens, table, 8, 8, &c, 0.1f, at(2), ldq, at(3),
                                                          (size_t)1 << 40, nullptr);
  printf("status %d\n", st);
  return 0;
}
