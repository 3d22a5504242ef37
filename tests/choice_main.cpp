// Prints the kernel that a call takes, for lines of: operation, SwiGLU, groups, rows, n_out, n_in, columns to a scale.
#include <cstdio>
#include <cstring>

#include "choice.h"

int main() {
    static const char *const q4[] = {"few", "16 halves", "16", "32", "64 halves", "64"};
    static const char *const bf16[] = {"128x64", "256x128 of 4", "256x128 of 8", "256x256", "few rows"};
    char op[16];
    int swiglu, groups, rows, n_out, n_in, scale;
    while (scanf("%15s %d %d %d %d %d %d", op, &swiglu, &groups, &rows, &n_out, &n_in, &scale) == 7) {
        if (!strcmp(op, "q4")) puts(q4[moe::q4_choice(swiglu, groups, rows, n_out, n_in, scale)]);
        else if (!strcmp(op, "linear")) puts(bf16[moe::grouped_choice(false, swiglu, groups, rows, n_out, n_in)]);
        else if (!strcmp(op, "dgrad")) puts(bf16[moe::grouped_choice(true, false, groups, rows, n_out, n_in)]);
        else if (!strcmp(op, "wgrad")) puts(moe::wgrad_256(groups, n_out, n_in) ? "256x256" : "128x128");
        else return 1;
    }
    return 0;
}
