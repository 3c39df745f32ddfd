// Host program for tests/test_pages_fill_host.py: prints, for 0 .. argv[1] copies sent, the parities of PaFill (qe_pages_fill.cuh).
#include <cstdio>
#include <cstdlib>
#include "qe_pages_fill.cuh"

int main(int argc, char** argv) {
  qe::PaFill f;
  for (int n = argc > 1 ? atoi(argv[1]) : 0; f.sent <= n; ++f.sent) printf("%u %u\n", f.empty(), f.landed());
}
