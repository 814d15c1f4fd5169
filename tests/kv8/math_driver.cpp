// Runs the 8-bit cache's arithmetic (csrc/ccb_kv8_math.h) on the host: reads
// binary records from stdin, writes results to stdout.  Modes:
//   e F   records of 4 floats (hi, lo, inv, s)  -> code byte of encode<F>
//   v F   records of 3 floats (x, inv, s)       -> code byte of encode_value<F>
//   b F   records of 1 float (a)                -> float block_scale<F>
//   w     records of 1 float                    -> uint32 weight_key
//   l     records of 2 int32 (len, capacity)    -> int32 checked_len
//   p     records of 2 int32 (page, numPages)   -> int32 checked_page
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "ccb_kv8_math.h"

template <int F>
static int run(char mode)
{
    float r[4];
    if (mode == 'e')
        while (fread(r, 4, 4, stdin) == 4) putchar(kv8::encode<F>(r[0], r[1], r[2], r[3]));
    else if (mode == 'v')
        while (fread(r, 4, 3, stdin) == 3) putchar(kv8::encode_value<F>(r[0], r[1], r[2]));
    else
        while (fread(r, 4, 1, stdin) == 1) {
            const float s = kv8::block_scale<F>(r[0]);
            fwrite(&s, 4, 1, stdout);
        }
    return 0;
}

int main(int argc, char** argv)
{
    if (argc < 2) return 2;
    const char mode = argv[1][0];
    if (mode == 'w') {
        float x;
        while (fread(&x, 4, 1, stdin) == 1) {
            const uint32_t k = kv8::weight_key(x);
            fwrite(&k, 4, 1, stdout);
        }
        return 0;
    }
    if (mode == 'l' || mode == 'p') {
        int32_t r[2];
        while (fread(r, 4, 2, stdin) == 2) {
            const int32_t v = mode == 'l' ? kv8::checked_len(r[0], r[1]) : kv8::checked_page(r[0], r[1]);
            fwrite(&v, 4, 1, stdout);
        }
        return 0;
    }
    if (argc < 3) return 2;
    return argv[2][0] == '0' ? run<kv8::kInt8>(mode) : run<kv8::kE4m3>(mode);
}
