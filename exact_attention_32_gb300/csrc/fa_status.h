// How the status words of several translation units' kernels make one (fa_get_device_status).  Host code without CUDA.
#pragma once

#include <initializer_list>

#include "fa.h"

// A call that failed counts for most, then a wait that gave up, since outputs are incomplete then and reading clears it; a bad page or
// sequence, whose part was left out, after both.
inline int fa_joined_status(const int *words, int n)
{
    int first = FA_OK;
    for (const int most : {static_cast<int>(FA_ERR_LAUNCH), static_cast<int>(FA_ERR_TIMEOUT)})
        for (int i = 0; i < n; ++i)
            if (words[i] == most) return most;
    for (int i = n - 1; i >= 0; --i)
        if (words[i] != FA_OK) first = words[i];
    return first;
}
