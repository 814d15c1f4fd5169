// Runs the move of codes to another block scale, eight at a time as the
// kernels do it (csrc/ccb_kv8_math.h, encode8_again), on the host: reads
// records of 10 floats (the codes' values, old scale, new scale) from stdin,
// writes 8 code bytes each.  Argument: the format.
#include <cstdio>

#include "ccb_kv8_math.h"

template <int F>
static int run()
{
    float r[10];
    while (fread(r, 4, 10, stdin) == 10) {
        uint32_t w[2];
        kv8::encode8_again<F>(r, r[8], 1.0f / r[9], r[9], w);
        for (int i = 0; i < 8; ++i) putchar((w[i / 4] >> (8 * (i % 4))) & 255);
    }
    return 0;
}

int main(int argc, char** argv)
{
    if (argc < 2) return 2;
    return argv[1][0] == '0' ? run<kv8::kInt8>() : run<kv8::kE4m3>();
}
