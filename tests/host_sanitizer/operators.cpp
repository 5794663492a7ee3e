// Host-side driver of the operators on rows of logits and of the block norm seam for the sanitizer build of the library:
// their workspace queries over valid and invalid sizes and the host validation of every entry point with arguments that
// it must reject before anything is launched. No GPU is needed. Exit status 0 when every call returned what it must.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "poet.h"

static int g_fail = 0;
#define EXPECT(cond)                                                     \
  do {                                                                   \
    if (!(cond)) {                                                       \
      std::fprintf(stderr, "FAILED line %d: %s\n", __LINE__, #cond);     \
      ++g_fail;                                                          \
    }                                                                    \
  } while (0)

// never dereferenced, far apart: validation fails first
template <class T = float> static T* at(int k) { return reinterpret_cast<T*>(uintptr_t(0x1000) + (uintptr_t(k) << 44)); }

int main() {
  const int32_t sizes[] = {-1, 0, 1, 2, 7, 8, 63, 1000, 32000, 32767, 32768, 65543, 131079, 131080, 1 << 24, (1 << 24) + 1,
                           INT32_MAX};
  for (int32_t T : sizes)
    for (int32_t V : sizes)
      for (int dt = -1; dt < 3; ++dt) {
        for (int32_t K : {-1, 0, 1, 20, 128, 129}) {
          const size_t b = poet_token_logprobs_workspace_bytes(T, V, dt, K);
          EXPECT(b == 0 || (T > 0 && V > 32768 && dt >= 0 && dt < 2 && K >= 0 && K <= 128) || (dt == 0 && V > 16384));
        }
        (void)poet_distill_workspace_bytes(T, V, dt);
        (void)poet_block_norm_workspace_bytes(T, V, dt);
      }
  for (int32_t T : {1, 2, 1000, 100000})
    for (int32_t d : {1, 7, 8, 512, 513, 4097, 8192, 16384})
      for (int32_t g : {0, 1, 2, 511, 100001}) EXPECT(poet_block_norm_workspace_bytes(T, d, g) > 0);

  poet_logits L{4, 100, 104, POET_BF16, 1.f};
  poet_teacher t{5, POET_DISTILL_RENORM, 1.f};
  int32_t* I = at<int32_t>(1);
  EXPECT(poet_token_logprobs(&L, nullptr, I, 0, nullptr, nullptr, at(2), at(3), nullptr, nullptr, at(4), nullptr, 0, nullptr,
                             0, nullptr) == POET_E_ARG);
  EXPECT(poet_token_logprobs(&L, at(5), I, 101, nullptr, nullptr, at(2), at(3), I, at(6), at(4), nullptr, 0, nullptr, 0,
                             nullptr) == POET_E_SHAPE);
  EXPECT(poet_token_logprobs_bwd(&L, at(5), I, at(4), at(2), nullptr, at(7), 99, nullptr) == POET_E_SHAPE);
  EXPECT(poet_distill(&L, &t, at(5), I, at(2), at(3), nullptr, at(8), at(4), nullptr, 0, nullptr, 0, nullptr) == POET_E_ARG);
  EXPECT(poet_distill_bwd(&L, &t, at(5), I, nullptr, nullptr, at(4), at(3), at(7), 104, nullptr) == POET_E_ARG);
  poet_logits wide{2000000000, 100, int64_t(1) << 40, POET_F32, 1.f};
  EXPECT(poet_token_logprobs_bwd(&wide, at(5), I, at(4), at(2), nullptr, at(7), 104, nullptr) == POET_E_UNSUPPORTED);
  poet_norm N{6, 100, 104, 104, 104, 104, POET_F32, POET_BF16, 2, 1.f, 1e-6f};
  EXPECT(poet_block_norm_fwd(&N, at(1), at(2), at(3), at(4), at(5), at(1), at(2), at(6), nullptr) == POET_E_ARG);
  EXPECT(poet_block_norm_fwd(&N, at(1), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, at(6), nullptr) == POET_E_ARG);
  EXPECT(poet_block_norm_bwd(&N, at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9), at(10), at(11), at(12),
                             at(13), at(14), 8, nullptr) == POET_E_WORKSPACE);
  N.T = INT32_MAX;
  N.ldh = int64_t(1) << 46;
  EXPECT(poet_block_norm_fwd(&N, at(1), at(2), at(3), at(4), at(5), at(7), at(8), at(6), nullptr) == POET_E_SHAPE);
  if (g_fail) std::fprintf(stderr, "%d checks failed\n", g_fail);
  else std::printf("operators sanitizer driver: all checks passed\n");
  return g_fail ? 1 : 0;
}
