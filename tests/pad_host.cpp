// Every chunk of rows of 1 to 80 elements at both halves of a word, with the loads checked: inside
// the row, words aligned, and the chunk's elements with zeros behind the row's end.
#include "pad.h"

#include <stdio.h>

int main()
{
    for (uint32_t dim = 1; dim <= 80; ++dim)
        for (uint32_t odd = 0; odd < 2; ++odd)
            for (uint32_t c = 0; c < (dim + 63) / 64 * 8; ++c) {
                uint32_t w[5], bad = 0;
                auto value = [](int64_t e) { return (uint32_t)(1000 + e) & 0xffff; };
                auto half = [&](int64_t e) {
                    bad |= e < 0 || e >= dim;
                    return (uint16_t)value(e);
                };
                auto word = [&](int64_t e) {
                    bad |= e < 0 || e + 1 >= dim || (e + odd) % 2;
                    return value(e) | value(e + 1) << 16;
                };
                zero::pad_load(w, c, dim, odd, word, half);
                zero::pad_shift(w, c, dim, odd);
                for (uint32_t i = 0; i < 8; ++i)
                    bad |= (w[i / 2] >> i % 2 * 16 & 0xffff) != (8 * c + i < dim ? value(8 * c + i) : 0);
                if (bad) {
                    printf("dim %u odd %u chunk %u\n", dim, odd, c);
                    return 1;
                }
            }
    puts("ok");
    return 0;
}
